"""Rotary append on the GPU: queries against the formula in 64 bits, keys and values bit for bit
against the plain append of the rotated keys, for every pool kind."""

import numpy as np
import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from chunk_ref import BF16_HALF, KINDS, assert_within, make_pool, rope_freqs_ref, rotate_ref

pytestmark = pytest.mark.gpu

RULES = {"plain": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=8.0),
         "banded": dict(scaling="banded", factor=8.0, original_len=8192, low=1.0, high=4.0),
         "yarn": dict(scaling="yarn", factor=16.0, original_len=4096, low=1.0, high=32.0)}


def _inputs(n, n_q, n_kv, dev, seed=0, fused=False):
    g = torch.Generator("cpu").manual_seed(seed)
    if fused:
        x = torch.randn(n, n_q + 2 * n_kv, 128, generator=g).bfloat16().to(dev)
        return x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    return tuple(torch.randn(n, h, 128, generator=g).bfloat16().to(dev) for h in (n_q, n_kv, n_kv))


def _check_queries(q, q_out, pos, rot, inter, rule):
    th, m = rope_freqs_ref(rot, 500000.0, **rule)
    x = q.double().cpu().numpy()
    y, size = rotate_ref(x, pos, th, m, rot, inter)
    # bf16 rounding; cos and sin off by 2^-21 (place in the turn 2^-24·2π, sincospif 2 ulp), products 2^-23
    assert_within(q_out.double().cpu().numpy(), y, BF16_HALF * np.abs(y) + 2.0 ** -20 * size + 1e-38, "q_out")
    rest = q_out[..., rot:].view(torch.int16)
    assert torch.equal(rest, q[..., rot:].contiguous().view(torch.int16))   # untouched dims keep their bits


@pytest.mark.parametrize("rule", sorted(RULES))
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (64, False), (66, False), (66, True), (2, False),
                                       (16, False), (126, False), (14, True)])
def test_queries_follow_the_formula(cuda_device, rule, rot, inter):
    if rule == "ntk" and rot == 2:
        pytest.skip("needs rot_dim >= 4")
    n, n_q, n_kv = 37, 5, 1
    q, k, v = _inputs(n, n_q, n_kv, cuda_device, rot)
    pos = np.random.default_rng(rot).integers(0, 1 << 24, n)
    pos[:3] = (0, (1 << 24) - 1, 131071)
    pool, _ = make_pool("bf16", 1, n_kv, 8, cuda_device)
    rope = kvd.Rope(rot, 500000.0, interleaved=inter, device=cuda_device, **RULES[rule])
    out = torch.empty_like(q)
    kvd.kvd_rope_append(pool.handle, 0, q, k, v, torch.tensor(pos, dtype=torch.int32, device=cuda_device), rope,
                        torch.arange(n, device=cuda_device), out)
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
    _check_queries(q, out, pos, rot, inter, RULES[rule])


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("slots", ["start_inside", "aligned", "scattered", "two_requests", "same_offset", "one"])
def test_append_equals_the_two_steps(cuda_device, kind, slots):
    """The pool's bytes are those of kvd_append_kv of the rotated keys, wherever the slots lie."""
    n, n_q, n_kv, blocks = 53, 3, 2, 20
    rng = np.random.default_rng(3)
    perm = rng.permutation(blocks)
    if slots == "one":
        n = 1
    run = {"start_inside": np.arange(5, 5 + n), "aligned": np.arange(n), "one": np.array([77])}
    if slots in run:
        flat = run[slots]
        slot = perm[flat // 16] * 16 + flat % 16
    elif slots == "scattered":
        slot = rng.permutation(blocks * 16)[:n]
    elif slots == "two_requests":
        flat = np.concatenate([np.arange(7, 7 + 20), np.arange(160 + 3, 160 + 3 + n - 20)])
        slot = perm[flat // 16] * 16 + flat % 16
    else:
        n = 17
        slot = perm[:n] * 16 + 9
    slot = slot.astype(np.int64)
    slot[n // 2] = -1   # a token without a slot
    q, k, v = _inputs(n, n_q, n_kv, cuda_device, 1, fused=True)
    pos = torch.arange(1000, 1000 + n, dtype=torch.int32, device=cuda_device)
    rope = kvd.Rope(128, 10000.0, device=cuda_device)
    sl = torch.tensor(slot, device=cuda_device)
    a, _ = make_pool(kind, 2, n_kv, blocks, cuda_device, fill=0)
    b, _ = make_pool(kind, 2, n_kv, blocks, cuda_device, fill=0)
    out = torch.empty(n, n_q, 128, dtype=torch.bfloat16, device=cuda_device)
    kvd.kvd_rope_append(a.handle, 1, q, k, v, pos, rope, sl, out)
    rotated = torch.empty(n, n_kv, 128, dtype=torch.bfloat16, device=cuda_device)
    scratch, _ = make_pool("bf16", 1, n_kv, blocks, cuda_device)
    kvd.kvd_rope_append(scratch.handle, 0, k, k, v, pos, rope, torch.full_like(sl, -1), rotated)
    kvd.kvd_append_kv(b.handle, 1, rotated, v.contiguous(), sl)
    assert torch.equal(a.mem, b.mem)
    assert (scratch.mem == 0xFF).all()
    assert kvd.kvd_get_device_error(a.handle) == kvd.KVD_OK


def test_in_place_strides_and_no_queries(cuda_device):
    n, n_q, n_kv = 40, 4, 2
    q, k, v = _inputs(n, n_q, n_kv, cuda_device, 5, fused=True)
    keep = q.clone()
    rope = kvd.Rope(96, 500000.0, device=cuda_device)
    pos = torch.arange(n, dtype=torch.int32, device=cuda_device)
    slot = torch.arange(n, device=cuda_device) + 16
    pool, _ = make_pool("bf16", 1, n_kv, 8, cuda_device, fill=0)
    kk, vv = k.clone(), v.clone()
    kvd.kvd_rope_append(pool.handle, 0, q, k, v, pos, rope, slot)    # into q itself, a slice of a wider tensor
    _check_queries(keep, q, np.arange(n), 96, False, {})
    assert torch.equal(k, kk) and torch.equal(v, vv)
    other, _ = make_pool("bf16", 1, n_kv, 8, cuda_device, fill=0)
    kvd.kvd_rope_append(other.handle, 0, None, k, v, pos, rope, slot)
    assert torch.equal(pool.mem, other.mem)


def test_bad_positions_and_slots_are_skipped(cuda_device):
    n, n_kv = 20, 1
    q, k, v = _inputs(n, 2, n_kv, cuda_device, 6)
    rope = kvd.Rope(128, 10000.0, device=cuda_device)
    pos = torch.arange(n, dtype=torch.int32)
    pos[3], pos[4] = -1, 1 << 24
    slot = torch.arange(n)
    slot[7] = 4 * 16
    pool, _ = make_pool("bf16", 1, n_kv, 4, cuda_device, fill=0)
    out = torch.full_like(q, 7.0)
    kvd.kvd_rope_append(pool.handle, 0, q, k, v, pos.to(cuda_device), rope, slot.to(cuda_device), out)
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_ERR_OOB
    assert (out[3:5] == 7.0).all() and not (out[7] == 7.0).any()
    from harness import read_record
    kt, vt = read_record(pool, 0, 0, 0)
    assert (kt[[3, 4, 7]] == 0).all() and (vt[[3, 4, 7]] == 0).all()
    assert torch.equal(vt[5], v[5, 0].cpu())


def test_captured_and_replayed(cuda_device):
    n, n_q, n_kv = 33, 4, 2
    q, k, v = _inputs(n, n_q, n_kv, cuda_device, 8)
    rope = kvd.Rope(128, 10000.0, device=cuda_device)
    pos = torch.arange(n, dtype=torch.int32, device=cuda_device)
    slot = torch.arange(n, device=cuda_device)
    pool, _ = make_pool("bf16", 1, n_kv, 4, cuda_device, fill=0)
    out = torch.empty_like(q)
    kvd.kvd_rope_append(pool.handle, 0, q, k, v, pos, rope, slot, out)
    want, mem = out.clone(), pool.mem.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.kvd_rope_append(pool.handle, 0, q, k, v, pos, rope, slot, out)
    out.zero_()
    pool.mem.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(pool.mem, mem)
    pos.add_(100)   # new positions in the same buffers
    graph.replay()
    torch.cuda.synchronize()
    th, m = rope_freqs_ref(128, 10000.0)
    y, size = rotate_ref(q.double().cpu().numpy(), np.arange(100, 100 + n), th, m, 128, False)
    assert_within(out.double().cpu().numpy(), y, BF16_HALF * np.abs(y) + 2.0 ** -20 * size + 1e-38, "replayed")
