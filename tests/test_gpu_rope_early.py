"""A decode step whose queries and keys are rotated first: with the append in the rotary call, and with the decode's
fused append, which lets the decode start early."""

import numpy as np
import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from chunk_ref import KINDS, make_pool, slots_of, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_rotated_keys_through_the_fused_append(cuda_device, kind):
    """Two layers a step, three steps: slots of -1 rotate q and (as q) k and write no pool, the decode appends the
    rotated keys and may pass the early-start flag behind them; pools and outputs equal those of the rotary append
    followed by a plain decode, bit for bit."""
    n_q, n_kv, layers = 16, 2, 2
    ctx = [900, 33, 2000, 1]
    total = [n + 3 for n in ctx]
    bt, nb = tables(total, 0, 3)
    g = torch.Generator("cpu").manual_seed(4)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_device)  # noqa: E731
    rope, btd = kvd.Rope(128, 10000.0, device=cuda_device), t(bt)
    pools = [make_pool(kind, layers, n_kv, nb, cuda_device, seed=1)[0] for _ in range(2)]
    for b, n in enumerate(ctx):
        k, v = (torch.randn(n, n_kv, 128, generator=g).bfloat16().to(cuda_device) for _ in range(2))
        for p in pools:
            for layer in range(layers):
                kvd.kvd_append_kv(p.handle, layer, k, v, t(slots_of(bt, b, 0, n)))
    nowhere = torch.full((4,), -1, dtype=torch.int64, device=cuda_device)
    ws = torch.empty(kvd.kvd_decode_workspace_bytes(pools[0].handle, n_q, 4, max(total))[1], dtype=torch.uint8,
                     device=cuda_device)
    for step in range(3):
        lens = [n + step + 1 for n in ctx]
        seq, pos = t(np.array(lens, np.int32)), t(np.array(lens, np.int32) - 1)
        slot = t(np.concatenate([slots_of(bt, b, n - 1, n) for b, n in enumerate(lens)]))
        x = [[torch.randn(4, h, 128, generator=g).bfloat16().to(cuda_device) for h in (n_q, n_kv, n_kv)]
             for _ in range(layers)]
        outs = []
        for early, p in zip((False, True), pools):
            got = [torch.zeros(4, n_q, 128, device=cuda_device) for _ in range(layers)]
            torch.cuda.synchronize()
            for layer, (q, k, v) in enumerate(x):
                rq, rk = torch.empty_like(q), torch.empty_like(k)
                if early:
                    kvd.kvd_rope_append(p.handle, layer, k, k, v, pos, rope, nowhere, rk)
                    kvd.kvd_rope_append(p.handle, layer, q, k, v, pos, rope, nowhere, rq)
                    kvd.kvd_decode_attn(p.handle, layer, rq, btd, seq, max(lens), ws, got[layer], k_new=rk, v_new=v,
                                        early_start=True)
                else:
                    kvd.kvd_rope_append(p.handle, layer, q, k, v, pos, rope, slot, rq)
                    kvd.kvd_decode_attn(p.handle, layer, rq, btd, seq, max(lens), ws, got[layer])
            outs.append(got)
        for a, b in zip(*outs):
            assert torch.equal(a, b)
        assert torch.equal(pools[0].mem, pools[1].mem)
    for p in pools:
        assert kvd.kvd_get_device_error(p.handle) == kvd.KVD_OK


def test_keys_rotated_in_place_without_an_append(cuda_device):
    n, n_kv = 300, 3
    g = torch.Generator("cpu").manual_seed(6)
    x = torch.randn(n, 9, 128, generator=g).bfloat16().to(cuda_device)
    k, v = x[:, 3:6], x[:, 6:]
    pool, _ = make_pool("bf16", 1, n_kv, 4, cuda_device)
    rope, pos = kvd.Rope(128, 10000.0, device=cuda_device), torch.arange(n, dtype=torch.int32, device=cuda_device)
    nowhere = torch.full((n,), -1, dtype=torch.int64, device=cuda_device)
    before, apart = x.clone(), torch.empty(n, n_kv, 128, dtype=torch.bfloat16, device=cuda_device)
    kvd.kvd_rope_append(pool.handle, 0, k, k, v, pos, rope, nowhere, apart)
    assert torch.equal(x, before)
    kvd.kvd_rope_append(pool.handle, 0, k, k, v, pos, rope, nowhere)
    assert torch.equal(k, apart) and torch.equal(x[:, :3], before[:, :3]) and torch.equal(v, before[:, 6:])
    assert (pool.mem == 0xFF).all() and kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
