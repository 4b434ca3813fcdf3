"""Compaction on the GPU: the new blocks' bytes are those of appending the retained tokens there."""

import numpy as np
import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from chunk_ref import KINDS, make_pool, slots_of, tables

pytestmark = pytest.mark.gpu


def _fill(pool, layers, k, v, slots, dev):
    for layer in range(layers):
        kvd.kvd_append_kv(pool.handle, layer, (k[layer]).to(dev), (v[layer]).to(dev), torch.from_numpy(slots).to(dev))


def _case(kind, lens, evict, dev, n_kv=2, layers=2, seed=0, width=0, host=0):
    rng = np.random.default_rng(seed)
    bt, nb = tables(lens, 0, seed, width)
    total = 2 * nb + 2
    new = np.full_like(bt, -1)
    perm = rng.permutation(np.arange(nb, total))
    at = 0
    for b, n in enumerate(lens):
        c = -(-n // 16)
        new[b, :c] = perm[at:at + c]
        at += c
    retain = ((rng.random((total, 16)) >= evict) << np.arange(16)).sum(1).astype(np.uint16)
    return rng, bt, new, nb, total, retain


def _run(pool, bt, lens, new, dev, retain=None, scores=None, stride=0):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    mask = None if retain is None else t(retain.view(np.int16))
    ws = torch.full((kvd.kvd_compact_workspace_bytes(pool.handle, len(lens), bt.shape[1]),), 0xEE, dtype=torch.uint8,
                    device=dev)
    new_lens = torch.full((len(lens),), -7, dtype=torch.int32, device=dev)
    ns = torch.full((len(lens), stride), 5.0, device=dev) if stride else None
    kvd.kvd_compact(pool.handle, t(bt), t(np.array(lens, np.int32)), t(new), new_lens, ws, retain_mask=mask,
                    scores=None if scores is None else t(scores), new_scores=ns)
    return new_lens.cpu().numpy(), mask, ns


@pytest.mark.parametrize("kind", sorted(set(KINDS) - {"mixed"}))
@pytest.mark.parametrize("evict", [0.0, 0.03, 0.5, 0.95])
def test_bytes_equal_an_append_of_the_retained(cuda_device, kind, evict):
    lens, layers, n_kv = [200, 1, 16, 33, 0, 517], 2, 3
    rng, bt, new, nb, total, retain = _case(kind, lens, evict, cuda_device, seed=int(evict * 100))
    pool, _ = make_pool(kind, layers, n_kv, total, cuda_device)
    want, _ = make_pool(kind, layers, n_kv, total, cuda_device)
    scores = rng.random((len(lens), 600)).astype(np.float32)
    kept = []
    for b, n in enumerate(lens):
        k, v = (torch.from_numpy(rng.standard_normal((layers, n, n_kv, 128))).bfloat16() for _ in range(2))
        s = slots_of(bt, b, 0, n)
        keep = np.array([(int(retain[x // 16]) >> (x % 16)) & 1 for x in s], bool)
        kept.append(np.nonzero(keep)[0])
        m = int(keep.sum())
        if n:
            _fill(pool, layers, k, v, s, cuda_device)
            _fill(want, layers, k, v, s, cuda_device)
        to = slots_of(new, b, 0, m)
        wm = want.mem.view(layers, total, -1)
        for j in range(-(-m // 16)):
            wm[:, int(new[b, j])] = 0
        if m:
            _fill(want, layers, k[:, keep], v[:, keep], to, cuda_device)
    new_lens, mask, ns = _run(pool, bt, lens, new, cuda_device, retain, scores, 555)
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
    assert new_lens.tolist() == [len(x) for x in kept]
    assert torch.equal(pool.mem, want.mem)          # old blocks and unused new ones as they were
    expect = retain.copy()
    for b, x in enumerate(kept):
        expect[new[b, :-(-len(x) // 16)]] = 0xFFFF
        row = np.zeros(555, np.float32)
        row[:len(x)] = scores[b, x]
        assert np.array_equal(ns[b].cpu().numpy(), row)
    assert np.array_equal(mask.cpu().numpy().view(np.uint16), expect)


def test_without_a_mask_it_forks(cuda_device):
    """A copy of a request that shares its source with another row of the call."""
    lens = [45, 45, 20]
    rng, bt, new, nb, total, _ = _case("bf16", lens, 0.0, cuda_device, seed=3)
    bt[1] = bt[0]
    pool, _ = make_pool("bf16", 1, 2, total, cuda_device)
    pool.mem.copy_(torch.randint(0, 256, pool.mem.shape, dtype=torch.uint8))
    before = pool.mem.clone()
    new_lens, _, _ = _run(pool, bt, lens, new, cuda_device)
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK and new_lens.tolist() == lens
    from harness import read_record
    ref = type("P", (), dict(mem=before, kv_dtype=pool.kv_dtype, record_bytes=8192, num_blocks=total, n_kv=2))()
    for b, n in enumerate(lens):
        for j in range(-(-n // 16)):
            m = min(16, n - 16 * j)
            for h in range(2):
                for x, y in zip(read_record(pool, 0, int(new[b, j]), h), read_record(ref, 0, int(bt[b, j]), h)):
                    assert torch.equal(x[:m].view(torch.int16), y[:m].view(torch.int16))
                    assert (x[m:] == 0).all()


def test_bad_ids_are_reported_and_not_written(cuda_device):
    lens = [64, 64]
    rng, bt, new, nb, total, _ = _case("bf16", lens, 0.0, cuda_device, seed=4)

    def run(bt, new, lens=lens):
        pool, _ = make_pool("bf16", 1, 1, total, cuda_device)
        src = torch.arange(nb, device=cuda_device, dtype=torch.uint8)[:, None].expand(nb, 8192)
        pool.mem.view(total, 8192)[:nb] = src
        got = _run(pool, bt, lens, new, cuda_device)[0]
        assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_ERR_OOB
        m = pool.mem.view(total, 8192).cpu()
        assert torch.equal(m[:nb], src.cpu())          # sources never written
        return got, m

    x = new.copy()
    x[0, 1], x[1, 3], x[0, 2] = total, -1, bt[1, 0]     # outside, outside, a source of the call
    got, m = run(bt, x)
    assert got.tolist() == lens and (m[int(new[0, 0])] == int(bt[0, 0])).all()
    x = new.copy()
    x[1, 2] = x[0, 0]                                    # the same new block twice
    got, m = run(bt, x)
    assert (m[int(new[0, 0])] == 0xFF).all()
    y = bt.copy()
    y[0, 1] = total + 5                                  # a bad source: its positions drop out
    got, m = run(y, new)
    assert got.tolist() == [48, 64]
    got, m = run(bt, new, [65, 64])                      # longer than its row
    assert got.tolist() == [0, 64]
    got, m = run(bt, np.ascontiguousarray(new[:, :3]))   # new rows too short: nothing copied
    assert got.tolist() == [0, 0] and (m[nb:] == 0xFF).all()


def test_host_tier_blocks(cuda_device):
    """Old and new blocks in either tier."""
    lens, layers, n_kv, nb = [100, 70], 2, 2, 12
    pool, _ = make_pool("fp8", layers, n_kv, nb, cuda_device)
    pool.attach_host_tier(14)
    ids = np.random.default_rng(5).permutation(26)
    bt, new = np.full((2, 7), -1, np.int32), np.full((2, 7), -1, np.int32)
    bt[0, :7], bt[1, :5], new[0, :7], new[1, :5] = ids[:7], ids[7:12], ids[12:19], ids[19:24]
    rng = np.random.default_rng(6)
    want, _ = make_pool("fp8", layers, n_kv, nb, cuda_device)
    want.attach_host_tier(14)
    for p in (pool, want):
        p.host_mem.fill_(0xFF)
    for b, n in enumerate(lens):
        k, v = (torch.from_numpy(rng.standard_normal((layers, n, n_kv, 128))).bfloat16() for _ in range(2))
        for p in (pool, want):
            _fill(p, layers, k, v, slots_of(bt, b, 0, n), cuda_device)
        for j in range(-(-n // 16)):
            i = int(new[b, j])
            torch.cuda.synchronize()
            if i < nb:
                want.mem.view(layers, nb, -1)[:, i] = 0
            else:
                want.host_mem.view(layers, 14, -1)[:, i - nb] = 0
        _fill(want, layers, k, v, slots_of(new, b, 0, n), cuda_device)
    got = _run(pool, bt, lens, new, cuda_device)[0]
    torch.cuda.synchronize()
    assert got.tolist() == lens and kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
    assert torch.equal(pool.mem, want.mem) and torch.equal(pool.host_mem, want.host_mem)


def test_captured_and_replayed(cuda_device):
    lens = [130, 60]
    rng, bt, new, nb, total, retain = _case("bf16", lens, 0.3, cuda_device, seed=7)
    pool, _ = make_pool("bf16", 3, 2, total, cuda_device)
    pool.mem.copy_(torch.randint(0, 256, pool.mem.shape, dtype=torch.uint8))
    start = pool.mem.clone()
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_device)  # noqa: E731
    a = [t(bt), t(np.array(lens, np.int32)), t(new), torch.zeros(2, dtype=torch.int32, device=cuda_device),
         torch.empty(kvd.kvd_compact_workspace_bytes(pool.handle, 2, bt.shape[1]), dtype=torch.uint8, device=cuda_device)]
    mask = t(retain.view(np.int16))
    kvd.kvd_compact(pool.handle, *a, retain_mask=mask)
    want, n = pool.mem.clone(), a[3].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kvd.kvd_compact(pool.handle, *a, retain_mask=mask)
    for _ in range(3):
        pool.mem.copy_(start)
        a[4].fill_(0xEE)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.mem, want) and torch.equal(a[3], n)


def test_a_prompt_an_eviction_and_the_next_step(cuda_device):
    """The operators in a row, as a server uses them: a prompt's chunks are rotated, appended and attended,
    slots are evicted, the cache is compacted, and a decode step and a further chunk over the dense blocks
    equal those over the masked ones."""
    n_q, n_kv, L = 8, 2, 2
    lens = [200, 77]
    total_lens = [n + 24 for n in lens]
    bt, nb = tables(total_lens, 0, 8)
    total = 2 * nb
    new = np.where(bt >= 0, bt + nb, -1).astype(np.int32)
    pool, _ = make_pool("bf16", L, n_kv, total, cuda_device)
    rope = kvd.Rope(128, 500000.0, device=cuda_device, scaling="banded", factor=8.0, original_len=8192, low=1.0, high=4.0)
    g = torch.Generator("cpu").manual_seed(1)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_device)  # noqa: E731
    ws = torch.empty(kvd.kvd_chunk_workspace_bytes(pool.handle, n_q, 2), dtype=torch.uint8, device=cuda_device)

    def step(layer, table, base, n_new, offset, retain):
        """n_new[b] tokens of every request appended behind base[b] slots at position offset[b]; attended."""
        n = sum(n_new)
        x = [torch.randn(n, h, 128, generator=g).bfloat16().to(cuda_device) for h in (n_q, n_kv, n_kv)]
        return x, attend(layer, table, base, n_new, offset, retain, x)

    def attend(layer, table, base, n_new, offset, retain, x):
        pos = np.concatenate([np.arange(o, o + m) for o, m in zip(offset, n_new)]).astype(np.int32)
        slot = np.concatenate([slots_of(table, b, s, s + m) for b, (s, m) in enumerate(zip(base, n_new))])
        q = torch.empty_like(x[0])
        kvd.kvd_rope_append(pool.handle, layer, *x, t(pos), rope, t(slot), q)
        out = torch.empty(q.shape, device=cuda_device)
        start = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        seq = t(np.array([s + m for s, m in zip(base, n_new)], np.int32))
        kvd.kvd_chunk_attn(pool.handle, layer, q, t(start), t(table), seq, ws, out, retain_mask=retain)
        return q, out, seq

    for layer in range(L):
        step(layer, bt, [0, 0], [150, 40], [0, 0], None)
        step(layer, bt, [150, 40], [50, 37], [150, 40], None)
    retain = ((np.random.default_rng(2).random((total, 16)) >= 0.2) << np.arange(16)).sum(1).astype(np.uint16)
    mask = t(retain.view(np.int16))
    new_lens = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    cws = torch.empty(kvd.kvd_compact_workspace_bytes(pool.handle, 2, bt.shape[1]), dtype=torch.uint8, device=cuda_device)
    kvd.kvd_compact(pool.handle, t(bt), t(np.array(lens, np.int32)), t(new), new_lens, cws, retain_mask=mask)
    dense = new_lens.tolist()
    assert 0 < dense[0] < lens[0]
    # the slots of the new tokens are kept in both rows
    full = mask.clone()
    for b in range(2):
        for p in range(lens[b], total_lens[b]):
            blk = int(bt[b, p // 16])
            full[blk] |= torch.tensor(np.array([1 << (p % 16)], np.uint16).view(np.int16)[0], device=cuda_device)
    full[nb:] = -1
    for layer in range(L):
        x, (q, masked, _) = step(layer, bt, lens, [20, 7], lens, full)
        _, compacted, seq = attend(layer, new, dense, [20, 7], lens, full, x)
        # two roundings of the weights (2^-8 each) of sums of values of magnitude below 6
        assert (masked - compacted).abs().max().item() <= 2 * 6 * 2.0 ** -8
        dq = q[[19, 26]]
        o = [torch.empty(2, n_q, 128, device=cuda_device) for _ in range(2)]
        for table, s, out in ((bt, t(np.array([lens[0] + 20, lens[1] + 7], np.int32)), o[0]), (new, seq, o[1])):
            _, n = kvd.kvd_decode_workspace_bytes(pool.handle, n_q, 2, 256)
            kvd.kvd_decode_attn(pool.handle, layer, dq.contiguous(), t(table), s, 256,
                                torch.empty(n, dtype=torch.uint8, device=cuda_device), out, retain_mask=full)
        assert (o[0] - o[1]).abs().max().item() <= 2 * 6 * 2.0 ** -8
        assert (o[1] - compacted[[19, 26]]).abs().max().item() <= 2 * 6 * 2.0 ** -8
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
