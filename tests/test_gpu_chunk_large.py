"""The forms that large calls take: a schedule that counts a unit's start and end (from eight tiles a CTA on), rotary
append with eight query heads or four KV heads a CTA, compaction with several (layer, head) pairs a CTA and more than
256 blocks a request."""

import numpy as np
import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from chunk_ref import BF16_HALF, KINDS, assert_within, make_pool, rope_freqs_ref, rotate_ref, slots_of
from harness import assert_out_close
from test_gpu_chunk import Case
from test_gpu_chunk_precision import reference
from test_gpu_compact import _case, _fill, _run

pytestmark = pytest.mark.gpu


def tiles_of(c):
    """Tiles of 64 positions over all units (request, KV head, ⌊256/g⌋ tokens)."""
    tq, n = 256 // (c.n_q // c.n_kv), 0
    for b, m in enumerate(c.lens):
        t = int(c.start[b + 1] - c.start[b])
        n += sum(-(-(m - t + min(i + tq, t)) // 64) for i in range(0, t, tq))
    return n * c.n_kv


def unit_cost(c, dev):
    """What the schedule adds to a unit: a tile for every eight a CTA has, six at most."""
    return min(6, tiles_of(c) // (8 * torch.cuda.get_device_properties(dev).multi_processor_count))


def check(c, dev, d=None, rows=slice(None)):
    first = c.run(d=d)
    out, lse = first
    ref, rlse, mass, size = reference(c, dev)
    tol = mass * (2 * 2.0 ** -16 * size + 2.0 ** -16 + 2.0 ** -19)   # as for short contexts in test_gpu_chunk_precision
    assert bool(((out.double() - ref).abs() <= tol)[rows].all())
    ok = torch.isneginf(lse) & torch.isneginf(rlse) | \
        ((lse.double() - rlse).abs() <= 2.0 ** -16 * size[..., 0] + 2.0 ** -20 * (1 + rlse.abs()))
    assert bool(ok[rows].all())
    assert_out_close(out[rows].double().cpu().numpy(), ref[rows].cpu().numpy())
    again = c.run(d=d)
    assert torch.equal(again[0], out) and torch.equal(again[1].view(torch.int32), lse.view(torch.int32))
    return out, lse


@pytest.mark.parametrize("kind,g,q_len,ctx,n_kv,cost", [
    ("bf16", 4, 512, 900, 8, 1), ("fp8", 4, 512, 2300, 8, 2), ("bf16", 7, 700, 1200, 8, 3), ("mixed", 8, 400, 3000, 8, 4),
    ("bf16", 5, 1000, 2000, 8, 5), ("bf16", 4, 1500, 2100, 8, 6), ("angle", 3, 1500, 3000, 8, 6)])
def test_prompts(cuda_device, kind, g, q_len, ctx, n_kv, cost):
    """Units of up to 256 rows, the warpgroups on 128 each; every value of a unit's cost."""
    c = Case(cuda_device, kind, g * n_kv, n_kv, [q_len], [q_len + ctx], seed=80 + cost)
    assert unit_cost(c, cuda_device) == cost
    check(c, cuda_device)
    assert kvd.kvd_get_device_error(c.pool.handle) == kvd.KVD_OK


@pytest.mark.parametrize("evict", [0.0, 0.2])
@pytest.mark.parametrize("kind,longest,cost", [("bf16", 1200, 1), ("fp8", 1200, 1), ("bf16", 6000, 5)])
def test_ragged_batches(cuda_device, kind, longest, cost, evict):
    """Single tokens, drafts and prompts in one call, units of one and of two row groups, T = 0 among them."""
    batch = 100
    rng = np.random.default_rng(batch + longest)
    q = rng.choice([0, 1, 1, 4, 30, 64, 65, 130], batch)
    lens = q + np.exp(rng.uniform(0, np.log(longest), batch)).astype(int)
    lens[:4] = q[:4] + longest
    c = Case(cuda_device, kind, 16, 4, q, lens, seed=90, evict=evict)
    assert unit_cost(c, cuda_device) == cost
    check(c, cuda_device)
    assert kvd.kvd_get_device_error(c.pool.handle) == kvd.KVD_OK


def test_bad_requests_among_many(cuda_device):
    """Lengths and row pairs that do not hold, in a batch whose schedule counts units: contained, and reported."""
    rng = np.random.default_rng(5)
    q = rng.integers(1, 40, 120)
    lens = q + rng.integers(0, 700, 120)
    c = Case(cuda_device, "bf16", 16, 4, q, lens, seed=91)
    assert unit_cost(c, cuda_device) >= 1
    d = c.device()
    bad_len, bad_rows = [0, 17, 18, 61, 119], [33, 90]
    for b in bad_len:
        d["lens"][b] = [-1, int(q[b]) - 1, 1 << 30][b % 3]
    keep = np.ones(int(c.start[-1]), bool)
    zero = np.zeros(int(c.start[-1]), bool)
    for b in bad_len:
        zero[c.start[b]:c.start[b + 1]] = True
    start = c.start.copy()
    for b in bad_rows:   # the pair of b falls, and that of the request after it begins elsewhere: behind every row
        start[b + 1] = c.start[-1] + 7
        keep[c.start[b]:c.start[b + 2]] = False
    d["start"].copy_(torch.from_numpy(start))
    keep &= ~zero
    rows = torch.from_numpy(np.nonzero(keep)[0]).to(cuda_device)
    out, lse = check(c, cuda_device, d=d, rows=rows)
    z = torch.from_numpy(np.nonzero(zero)[0]).to(cuda_device)
    assert bool((out[z] == 0).all()) and bool(torch.isneginf(lse[z]).all())
    for b in bad_rows:
        assert bool((out[c.start[b]:c.start[b + 2]] == 9).all())
    assert kvd.kvd_get_device_error(c.pool.handle) == kvd.KVD_ERR_OOB


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("n_q,n_kv", [(24, 3), (28, 5), (24, 8), (25, 1)])
def test_rotary_append_of_a_prompt(cuda_device, kind, n_q, n_kv):
    """4,099 tokens that start inside a block, two requests, tokens without a slot: the pool's bytes are those of
    kvd_append_kv of the rotated keys.  25 and 28 query heads leave a last CTA of one and four, 3 and 5 KV heads one of
    three and one."""
    n, rot = 4099, 96
    per_cta = -(-n // 16) + 1
    assert per_cta * -(-n_q // 8) >= 4 * torch.cuda.get_device_properties(cuda_device).multi_processor_count
    blocks = 2 * (-(-n // 16) + 2)
    perm = np.random.default_rng(7).permutation(blocks)
    flat = np.concatenate([np.arange(5, 5 + 3000), np.arange(3200 + 9, 3200 + 9 + n - 3000)])
    slot = (perm[flat // 16] * 16 + flat % 16).astype(np.int64)
    slot[[0, 77, 3001, n - 1]] = -1
    g = torch.Generator("cpu").manual_seed(9)
    x = torch.randn(n, n_q + 2 * n_kv, 128, generator=g).bfloat16().to(cuda_device)
    q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    pos = torch.arange(120000, 120000 + n, dtype=torch.int32, device=cuda_device)
    rope = kvd.Rope(rot, 500000.0, device=cuda_device)
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
    alone, _ = make_pool(kind, 2, n_kv, blocks, cuda_device, fill=0)
    kvd.kvd_rope_append(alone.handle, 1, None, k, v, pos, rope, sl)
    assert torch.equal(a.mem, alone.mem)
    theta, m = rope_freqs_ref(rot, 500000.0)
    for got, src in ((out, q), (rotated, k)):
        y, size = rotate_ref(src.double().cpu().numpy(), pos.cpu().numpy(), theta, m, rot, False)
        assert_within(got.double().cpu().numpy(), y, BF16_HALF * np.abs(y) + 2.0 ** -20 * size + 1e-38, "rotated")
        assert torch.equal(got[..., rot:].view(torch.int16), src[..., rot:].contiguous().view(torch.int16))
    assert kvd.kvd_get_device_error(a.handle) == kvd.KVD_OK


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_rotary_append_of_a_prompt_over_both_tiers(cuda_device, kind):
    """Blocks in host memory get the bytes that they would get in the pool."""
    n, n_q, n_kv, blocks = 4099, 24, 5, 130
    perm = np.random.default_rng(8).permutation(2 * blocks)
    flat = np.arange(11, 11 + n)
    slot = (perm[flat // 16] * 16 + flat % 16).astype(np.int64)
    g = torch.Generator("cpu").manual_seed(10)
    q, k, v = (torch.randn(n, h, 128, generator=g).bfloat16().to(cuda_device) for h in (n_q, n_kv, n_kv))
    pos = torch.arange(n, dtype=torch.int32, device=cuda_device)
    rope, sl = kvd.Rope(128, 10000.0, device=cuda_device), torch.tensor(slot, device=cuda_device)
    one, _ = make_pool(kind, 1, n_kv, 2 * blocks, cuda_device, fill=0)
    two, _ = make_pool(kind, 1, n_kv, blocks, cuda_device, fill=0)
    two.attach_host_tier(blocks)
    two.host_mem.fill_(0)
    for p in (one, two):
        kvd.kvd_rope_append(p.handle, 0, q, k, v, pos, rope, sl, torch.empty_like(q))
    torch.cuda.synchronize()
    assert torch.equal(one.mem.cpu(), torch.cat([two.mem.cpu(), two.host_mem]))
    assert kvd.kvd_get_device_error(two.handle) == kvd.KVD_OK


@pytest.mark.parametrize("kind", sorted(set(KINDS) - {"mixed"}))
@pytest.mark.parametrize("evict", [0.0, 0.1])
def test_compaction_of_long_requests(cuda_device, kind, evict):
    """313 and 257 blocks, more than a pass of the ranks; 15 (layer, head) pairs for eight CTAs a block."""
    lens, layers, n_kv = [5000, 4111], 5, 3
    rng, bt, new, nb, total, retain = _case(kind, lens, evict, cuda_device, seed=11)
    pool, _ = make_pool(kind, layers, n_kv, total, cuda_device)
    want, _ = make_pool(kind, layers, n_kv, total, cuda_device)
    scores = rng.random((2, 5000)).astype(np.float32)
    kept = []
    for b, n in enumerate(lens):
        k, v = (torch.from_numpy(rng.standard_normal((layers, n, n_kv, 128), dtype=np.float32)).bfloat16() for _ in range(2))
        s = slots_of(bt, b, 0, n)
        keep = ((retain[s // 16].astype(np.int64) >> (s % 16)) & 1).astype(bool)
        kept.append(np.nonzero(keep)[0])
        m = int(keep.sum())
        for p in (pool, want):
            _fill(p, layers, k, v, s, cuda_device)
        want.mem.view(layers, total, -1)[:, torch.from_numpy(new[b, :-(-m // 16)].astype(np.int64)).to(cuda_device)] = 0
        _fill(want, layers, k[:, keep], v[:, keep], slots_of(new, b, 0, m), cuda_device)
    new_lens, mask, ns = _run(pool, bt, lens, new, cuda_device, retain, scores, 4800)
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
    assert new_lens.tolist() == [len(x) for x in kept]
    assert torch.equal(pool.mem, want.mem)
    expect = retain.copy()
    for b, x in enumerate(kept):
        expect[new[b, :-(-len(x) // 16)]] = 0xFFFF
        row = np.zeros(4800, np.float32)
        row[:min(len(x), 4800)] = scores[b, x][:4800]
        assert np.array_equal(ns[b].cpu().numpy(), row)
    assert np.array_equal(mask.cpu().numpy().view(np.uint16), expect)
