"""Chunk attention on the GPU against the plain form in 64 bits over the oracle's pool."""

import numpy as np
import pytest
import torch

import oracle
import paged_gqa_decode_kvd_gb300 as kvd
from chunk_ref import KINDS, assert_within, chunk_ref, make_oracle, make_pool, slots_of, tables

pytestmark = pytest.mark.gpu
BF16 = sorted(KINDS)


class Case:
    def __init__(self, dev, kind, n_q, n_kv, q_lens, lens, seed=0, evict=0.0, factor=1.0, spare=3, layers=1):
        rng = np.random.default_rng(seed)
        self.kind, self.n_q, self.n_kv, self.lens, self.dev = kind, n_q, n_kv, list(lens), dev
        self.bt, self.nb = tables(lens, spare, seed)
        self.pool, fmt = make_pool(kind, layers, n_kv, self.nb, dev, seed=seed)
        self.opool = make_oracle(kind, n_kv, self.nb, fmt)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            k = torch.from_numpy(rng.standard_normal((n, n_kv, 128)) * factor).bfloat16()
            v = torch.from_numpy(rng.standard_normal((n, n_kv, 128))).bfloat16()
            s = slots_of(self.bt, b, 0, n)
            kvd.kvd_append_kv(self.pool.handle, layers - 1, k.to(dev), v.to(dev), torch.from_numpy(s).to(dev))
            assert self.opool.append(k.float().numpy(), v.float().numpy(), s) == 0
        self.layer = layers - 1
        self.start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.q = torch.from_numpy(rng.standard_normal((int(self.start[-1]), n_q, 128))).bfloat16()
        self.retain = None
        if evict:
            keep = rng.random((self.nb, 16)) >= evict
            self.retain = (keep << np.arange(16)).sum(1).astype(np.uint16)

    def device(self):
        dev = self.dev
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        return dict(q=self.q.to(dev), start=t(self.start), bt=t(self.bt), lens=t(np.array(self.lens, np.int32)),
                    retain=None if self.retain is None else t(self.retain.view(np.int16)))

    def run(self, out_dtype=torch.float32, scale=None, retain=True, d=None, stream=None):
        d = d or self.device()
        ws = torch.empty(kvd.kvd_chunk_workspace_bytes(self.pool.handle, self.n_q, len(self.lens)), dtype=torch.uint8,
                         device=self.dev)
        out = torch.full(d["q"].shape, 9.0, dtype=out_dtype, device=self.dev)
        lse = torch.full(d["q"].shape[:2], 9.0, dtype=torch.float32, device=self.dev)
        kvd.kvd_chunk_attn(self.pool.handle, self.layer, d["q"], d["start"], d["bt"], d["lens"], ws, out,
                           retain_mask=d["retain"] if retain else None, softmax_scale=scale, lse_out=lse, stream=stream)
        return out, lse

    def reference(self, scale=None):
        k, v = self.opool.values()
        q = self.q.double().numpy()
        if self.kind == "angle":
            q = oracle.angle_query(self.q.float().numpy())
        return chunk_ref(k, v, q, self.start, self.bt, self.lens, self.retain, 128 ** -0.5 if scale is None else scale,
                         lowbit=KINDS[self.kind][1] > 0)

    def check(self, out_dtype=torch.float32, scale=None):
        out, lse = self.run(out_dtype, scale)
        ref, rlse, tol, ltol = self.reference(scale)
        assert kvd.kvd_get_device_error(self.pool.handle) == kvd.KVD_OK
        assert_within(lse.double().cpu().numpy(), rlse, ltol, "lse")
        assert_within(out.double().cpu().numpy(), ref, tol, "out")


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8])
def test_kinds_and_groups(cuda_device, kind, g):
    Case(cuda_device, kind, 2 * g, 2, [5, 1, 33], [70, 1, 161], seed=g).check()


@pytest.mark.parametrize("q_len,ctx", [(1, 0), (1, 15), (1, 16), (1, 63), (1, 64), (1, 1000), (2, 0), (16, 0), (17, 48),
                                       (64, 0), (64, 1), (65, 63), (100, 500), (128, 0), (129, 127), (200, 1)])
@pytest.mark.parametrize("n_q,n_kv", [(4, 1), (8, 1), (7, 1)])
def test_lengths(cuda_device, q_len, ctx, n_q, n_kv):
    Case(cuda_device, "bf16", n_q, n_kv, [q_len], [q_len + ctx], seed=q_len + ctx).check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "mixed", "int4"])
def test_ragged_batch_with_evictions(cuda_device, kind):
    q_lens = [1, 0, 37, 4, 90, 1, 2, 300]
    lens = [513, 100, 37, 260, 333, 1, 70, 301]
    Case(cuda_device, kind, 8, 2, q_lens, lens, seed=5, evict=0.3, factor=2.0).check(torch.bfloat16)


@pytest.mark.parametrize("batch", [150, 600])
def test_many_short_requests(cuda_device, batch):
    rng = np.random.default_rng(batch)
    q = rng.integers(0, 4, batch)
    Case(cuda_device, "bf16", 4, 2, q, q + rng.integers(0, 40, batch), seed=1).check()


def test_a_long_context_is_split(cuda_device):
    Case(cuda_device, "bf16", 4, 1, [3], [20011], seed=2).check()
    Case(cuda_device, "fp8", 8, 1, [17], [9001], seed=3).check()


def test_all_evicted_and_partly_empty_rows(cuda_device):
    c = Case(cuda_device, "bf16", 4, 2, [20, 20], [52, 52], seed=4)
    c.retain = np.full(c.nb, 0xFFFF, np.uint16)
    c.retain[c.bt[0, :4]] = 0            # nothing of request 0 is left
    c.retain[c.bt[1, :2]] = 0            # request 1 starts at position 40: its first rows see nothing
    c.retain[c.bt[1, 2]] = 0xFF00
    out, lse = c.run()
    assert (out[:20] == 0).all() and torch.isinf(lse[:20]).all()
    assert (out[20:28] == 0).all() and torch.isinf(lse[20:28]).all() and (lse[20:28] < 0).all()
    c.check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(cuda_device, scale):
    Case(cuda_device, "bf16", 4, 1, [30], [190], seed=6).check(scale=scale)


def test_large_logits(cuda_device):
    """Keys 60 times larger: the maximum moves by hundreds along the row and most weights vanish."""
    Case(cuda_device, "bf16", 4, 1, [70], [400], seed=7, factor=60.0).check()
    Case(cuda_device, "fp8", 8, 1, [9], [400], seed=8, factor=60.0).check()


def test_masked_slots_may_hold_anything(cuda_device):
    """NaN and infinities in evicted slots, behind the last position and in later new tokens."""
    c = Case(cuda_device, "bf16", 4, 1, [40], [100], seed=9, evict=0.2)
    ref, rlse, tol, ltol = c.reference()
    bad = torch.full((1, 1, 128), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    for p in range(112):
        blk, t = int(c.bt[0, p // 16]), p % 16
        if p >= 100 or not (int(c.retain[blk]) >> t) & 1:
            x = bad if p % 2 else torch.full_like(bad, float("inf"))
            kvd.kvd_append_kv(c.pool.handle, 0, x, x, torch.tensor([blk * 16 + t], device=cuda_device))
    out, lse = c.run()
    assert_within(out.double().cpu().numpy(), ref, tol, "out")
    assert_within(lse.double().cpu().numpy(), rlse, ltol, "lse")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_value_reaches_its_own_rows_only(cuda_device, value):
    """A non-finite V of new token 23 changes rows 23 and later, in that dim, and no earlier row."""
    c = Case(cuda_device, "bf16", 4, 1, [40], [100], seed=10)
    ref, rlse, tol, ltol = c.reference()
    pos = 60 + 23
    blk, t = int(c.bt[0, pos // 16]), pos % 16
    k, v = (torch.from_numpy(x[blk, :, t].copy()).bfloat16()[None].to(cuda_device) for x in c.opool.values())
    v[0, 0, 77] = value
    kvd.kvd_append_kv(c.pool.handle, 0, k, v, torch.tensor([blk * 16 + t], device=cuda_device))
    out, lse = (x.double().cpu().numpy() for x in c.run())
    assert_within(out[:23], ref[:23], tol[:23], "earlier rows")
    hit = out[23:, :, 77]
    assert np.isnan(hit).all() if np.isnan(value) else (hit == value).all()
    rest = np.delete(out[23:], 77, axis=2)
    assert_within(rest, np.delete(ref[23:], 77, axis=2), np.delete(tol[23:], 77, axis=2), "other dims")
    assert_within(lse, rlse, ltol, "lse")


@pytest.mark.parametrize("q_len,n_q", [(40, 4), (20, 1)])
@pytest.mark.parametrize("kind", ["fp8", "angle", "mixed", "int4", "int2"])
def test_masked_slots_of_any_format_may_hold_anything(cuda_device, kind, q_len, n_q):
    """NaN and infinities in evicted slots and behind the last position, in tiles with and without new tokens."""
    c = Case(cuda_device, kind, n_q, 1, [q_len], [300], seed=29, evict=0.2)
    ref, rlse, tol, ltol = c.reference()
    bad = torch.full((1, 1, 128), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    for p in range(304):
        blk, t = int(c.bt[0, p // 16]), p % 16
        if p >= 300 or not (int(c.retain[blk]) >> t) & 1:
            x = bad if p % 2 else torch.full_like(bad, float("inf"))
            kvd.kvd_append_kv(c.pool.handle, 0, x, x, torch.tensor([blk * 16 + t], device=cuda_device))
    out, lse = c.run()
    assert_within(out.double().cpu().numpy(), ref, tol, "out")
    assert_within(lse.double().cpu().numpy(), rlse, ltol, "lse")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n_q", [1, 4])
@pytest.mark.parametrize("kind", ["fp8", "angle", "mixed", "int4"])
def test_a_bad_value_of_any_format_spares_earlier_rows(cuda_device, kind, n_q, value):
    """A non-finite V of new token 23 reaches rows 23 and later and no earlier row; the logits do not know of it."""
    c = Case(cuda_device, kind, n_q, 1, [40], [100], seed=30)
    ref, rlse, tol, ltol = c.reference()
    pos = 60 + 23
    blk, t = int(c.bt[0, pos // 16]), pos % 16
    good = torch.from_numpy(np.random.default_rng(31).standard_normal((1, 1, 128))).bfloat16().to(cuda_device)
    v = good.clone()
    v[0, 0, 77] = value
    slot = np.array([blk * 16 + t])
    kvd.kvd_append_kv(c.pool.handle, 0, good, v, torch.from_numpy(slot).to(cuda_device))
    assert c.opool.append(good.float().cpu().numpy(), good.float().cpu().numpy(), slot) == 0
    ref, rlse, tol, ltol = c.reference()
    out, lse = (x.double().cpu().numpy() for x in c.run())
    assert_within(out[:23], ref[:23], tol[:23], "earlier rows")
    assert_within(lse, rlse, ltol, "lse")
    # (a low-bit record is finite whatever it is given: codes are clamped, and its scale and zero saturate in 16 bits)
    assert kind == "int4" or not np.isfinite(out[23:, :, 77]).any()


@pytest.mark.parametrize("kind,n_q", [("fp8", 4), ("fp8", 1), ("angle", 4)])
def test_a_bad_cached_value_reaches_every_row(cuda_device, kind, n_q):
    """An infinity in the cache ahead of the new tokens makes an 8-bit record's scale infinite: NaN in all rows."""
    c = Case(cuda_device, kind, n_q, 1, [40], [300], seed=32)
    blk, t = int(c.bt[0, 70 // 16]), 70 % 16
    v = torch.ones((1, 1, 128), dtype=torch.bfloat16, device=cuda_device)
    v[0, 0, 5] = float("inf")
    kvd.kvd_append_kv(c.pool.handle, 0, torch.zeros_like(v), v, torch.tensor([blk * 16 + t], device=cuda_device))
    out, lse = (x.double().cpu().numpy() for x in c.run())
    assert np.isnan(out).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "mixed"])
@pytest.mark.parametrize("q_lens,lens,n_q", [([1], [3], 1), ([1, 4, 2], [7, 60, 700], 4), ([100], [130], 8), ([128], [900], 8)])
def test_few_rows_keep_the_weights_precision(cuda_device, kind, q_lens, lens, n_q):
    """Up to 1,024 rows a weight is the sum of two bf16: off by 2^-9 · 2^-9 of itself.  Its logit, an fp32 sum of 128
    products and a multiplication, adds less than 2^-17 of it at |l| < 16, the fp32 sums over 900 positions less than
    2^-16 together: 2^-15 of the weighted mean of |v| bounds them all (a weight of 8 bits alone would be off by 2^-9)."""
    c = Case(cuda_device, kind, n_q, 1, q_lens, lens, seed=33)
    assert sum(q_lens) * n_q <= 1024
    out, _ = c.run()
    ref = c.reference()[0]
    k, v = c.opool.values()
    size = chunk_ref(k, np.abs(v), c.q.double().numpy(), c.start, c.bt, c.lens, None, 128 ** -0.5)[0]
    assert (np.abs(out.double().cpu().numpy() - ref) <= 2.0 ** -15 * size).all()


def test_a_nan_query_stays_in_its_row(cuda_device):
    c = Case(cuda_device, "bf16", 4, 1, [10], [100], seed=11)
    c.q[4, 2, 5] = float("nan")
    out, lse = (x.double().cpu().numpy() for x in c.run())
    q = c.q.clone()
    c.q = torch.nan_to_num(q)
    ref, rlse, tol, ltol = c.reference()
    assert np.isnan(out[4, 2]).all() and np.isnan(lse[4, 2])
    keep = np.ones((10, 4), bool)
    keep[4, 2] = False
    assert_within(out[keep], ref[keep], tol[keep], "other rows")


def test_shared_blocks(cuda_device):
    """Two requests share their prompt's blocks."""
    c = Case(cuda_device, "bf16", 4, 2, [5, 20], [101, 60], seed=12)
    c.bt[1, :3] = c.bt[0, :3]
    c.check()


def test_rows_outside_stay_as_they_are(cuda_device):
    c = Case(cuda_device, "bf16", 4, 2, [6, 9], [40, 50], seed=13)
    c.q = torch.cat([c.q, torch.randn(5, 4, 128).bfloat16()])
    c.start = c.start + 2                     # rows 0, 1 and the last 3 belong to no request
    d = c.device()
    out, lse = c.run(d=d)
    assert (out[:2] == 9).all() and (out[17:] == 9).all() and (lse[:2] == 9).all() and (lse[17:] == 9).all()
    c.q = c.q[:17]
    ref, rlse, tol, ltol = c.reference()
    assert_within(out[2:17].double().cpu().numpy(), ref[2:], tol[2:], "out")


def test_bad_requests_are_reported_and_contained(cuda_device):
    c = Case(cuda_device, "bf16", 4, 2, [4, 4, 4, 4, 4], [64, 64, 64, 64, 64], seed=14)
    ref, rlse, tol, ltol = c.reference()
    d = c.device()

    def run(**kw):
        out, lse = c.run(d={**d, **kw})
        assert kvd.kvd_get_device_error(c.pool.handle) == kvd.KVD_ERR_OOB
        return out.double().cpu().numpy(), lse.cpu().numpy()

    good = [0, 1, 3, 4]
    rows = np.concatenate([np.arange(4 * b, 4 * b + 4) for b in good])
    for n in (-1, 3, 65, 2 ** 31 - 1):       # shorter than its new tokens, longer than its table
        lens = d["lens"].clone()
        lens[2] = n
        out, lse = run(lens=lens)
        assert (out[8:12] == 0).all() and np.isneginf(lse[8:12]).all()
        assert_within(out[rows], ref[rows], tol[rows], "others")
    start = d["start"].clone()
    start[3] = 100                            # request 2 ends behind the rows; request 3 starts there
    out, lse = run(start=start)
    assert (out[8:16] == 9).all()
    assert_within(out[:8], ref[:8], tol[:8], "others")
    assert_within(out[16:], ref[16:], tol[16:], "others")
    bt = d["bt"].clone()
    bt[2, 1], bt[2, 2] = c.nb, -5             # positions 16 .. 47 of request 2 drop out
    out, lse = run(bt=bt)
    c.retain = np.full(c.nb, 0xFFFF, np.uint16)
    c.retain[c.bt[2, 1:3]] = 0
    ref2, _, tol2, _ = c.reference()
    assert_within(out, ref2, tol2, "without the bad blocks")


def test_layers_streams_and_repeats(cuda_device):
    """Another layer, another stream, the same bits every time."""
    c = Case(cuda_device, "fp8", 8, 2, [50, 3, 200], [50, 900, 412], seed=15, layers=3)
    c.check()
    first = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = c.run()
    s.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    for _ in range(5):
        for a, b in zip(first, c.run()):
            assert torch.equal(a, b)


def test_two_calls_at_once(cuda_device):
    """Two streams, a workspace each."""
    a = Case(cuda_device, "bf16", 8, 2, [300], [700], seed=16)
    b = Case(cuda_device, "bf16", 4, 2, [5, 60], [2000, 60], seed=17)
    want = a.run(), b.run()
    torch.cuda.synchronize()
    da, db = a.device(), b.device()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s):
            x = a.run(d=da)
        with torch.cuda.stream(t):
            y = b.run(d=db)
        torch.cuda.synchronize()
        for got, ref in ((x, want[0]), (y, want[1])):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_captured_with_new_lengths(cuda_device):
    """One captured call serves other lengths and tables written into its buffers."""
    c = Case(cuda_device, "bf16", 4, 2, [30, 10], [230, 150], seed=18)
    d = c.device()
    ws = torch.empty(kvd.kvd_chunk_workspace_bytes(c.pool.handle, 4, 2), dtype=torch.uint8, device=cuda_device)
    out, lse = torch.zeros(40, 4, 128, device=cuda_device), torch.zeros(40, 4, device=cuda_device)

    def call():
        kvd.kvd_chunk_attn(c.pool.handle, 0, d["q"], d["start"], d["bt"], d["lens"], ws, out, lse_out=lse)

    call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for q_lens, lens in (([30, 10], [230, 150]), ([1, 39], [200, 39]), ([40, 0], [41, 3])):
        c.start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        c.lens = lens
        d["start"].copy_(torch.from_numpy(c.start))
        d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        ref, rlse, tol, ltol = c.reference()
        assert_within(out.double().cpu().numpy(), ref, tol, "out")
        assert_within(lse.double().cpu().numpy(), rlse, ltol, "lse")


@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_host_tier(cuda_device, kind, staged):
    """Blocks in host memory give the result of the same blocks in the pool."""
    c = Case(cuda_device, kind, 8, 2, [20, 5], [300, 170], seed=19)
    want = c.run()
    pool, _ = make_pool(kind, 1, 2, c.nb, cuda_device)
    pool.attach_host_tier(c.nb, staged=staged)
    move = np.random.default_rng(0).random(c.nb) < 0.4
    ids = np.arange(c.nb, dtype=np.int32)
    to = np.where(move, ids + c.nb, ids)
    rec = pool.record_bytes * 2
    src = c.pool.mem.view(c.nb, rec).cpu()
    host = pool.host_mem.view(c.nb, rec)
    host[torch.from_numpy(move)] = src[torch.from_numpy(move)]
    pool.mem.view(c.nb, rec)[torch.from_numpy(~move).to(cuda_device)] = src[torch.from_numpy(~move)].to(cuda_device)
    kvd.kvd_tier_prefetch(pool.handle, 0)
    c.bt = np.where(c.bt >= 0, to[c.bt], -1).astype(np.int32)
    c.pool = pool
    got = c.run()
    torch.cuda.synchronize()
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_one_token_agrees_with_the_decode(cuda_device):
    c = Case(cuda_device, "bf16", 8, 2, [1, 1], [333, 40], seed=20, evict=0.1)
    out, lse = c.run()
    d = c.device()
    _, n = kvd.kvd_decode_workspace_bytes(c.pool.handle, 8, 2, 333)
    o, z = torch.empty_like(out), torch.empty_like(lse)
    kvd.kvd_decode_attn(c.pool.handle, 0, d["q"], d["bt"], d["lens"], 333,
                        torch.empty(n, dtype=torch.uint8, device=cuda_device), o, retain_mask=d["retain"], lse_out=z)
    _, _, tol, ltol = c.reference()
    assert_within(out.double().cpu().numpy(), o.double().cpu().numpy(), 2 * tol, "out")
    assert_within(lse.double().cpu().numpy(), z.double().cpu().numpy(), 2 * ltol, "lse")


def run_many_rows(c):
    """The call with rows behind the last request, more than 1,024 in all: those stay as they were."""
    d, n = c.device(), c.q.shape[0]
    d["q"] = torch.cat([d["q"], torch.full((1024 // c.n_q + 1, c.n_q, 128), float("nan"), dtype=torch.bfloat16, device=c.dev)])
    out, lse = c.run(d=d)
    assert (out[n:] == 9.0).all() and (lse[n:] == 9.0).all()
    return out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()


def check_many_rows(c):
    out, lse = run_many_rows(c)
    ref, rlse, tol, ltol = c.reference()
    assert kvd.kvd_get_device_error(c.pool.handle) == kvd.KVD_OK
    assert_within(lse, rlse, ltol, "lse")
    assert_within(out, ref, tol, "out")


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("g", [1, 3, 4, 7, 8])
def test_many_rows_kinds_and_groups(cuda_device, kind, g):
    check_many_rows(Case(cuda_device, kind, 2 * g, 2, [33, 1, 70], [97, 40, 133], seed=40 + g))


@pytest.mark.parametrize("q_len,ctx", [(1, 0), (1, 63), (1, 64), (1, 1000), (16, 0), (64, 0), (65, 63), (200, 511)])
@pytest.mark.parametrize("n_q", [4, 7])
def test_many_rows_lengths(cuda_device, q_len, ctx, n_q):
    check_many_rows(Case(cuda_device, "bf16", n_q, 1, [q_len], [q_len + ctx], seed=50 + q_len))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "mixed", "int4", "angle"])
def test_many_rows_ragged_with_evictions(cuda_device, kind):
    check_many_rows(Case(cuda_device, kind, 8, 2, [1, 0, 37, 4, 90, 1, 2, 300], [513, 100, 37, 260, 333, 1, 70, 301], seed=60,
                         evict=0.3, factor=2.0))
    check_many_rows(Case(cuda_device, kind, 4, 1, [3, 5], [9000, 4000], seed=61))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("kind,n_q", [("bf16", 1), ("bf16", 4), ("fp8", 1), ("fp8", 4), ("angle", 4), ("mixed", 4)])
def test_many_rows_a_bad_value_spares_earlier_rows(cuda_device, kind, n_q, value):
    c = Case(cuda_device, kind, n_q, 1, [40], [100], seed=62)
    pos = 60 + 23
    blk, t = int(c.bt[0, pos // 16]), pos % 16
    good = torch.from_numpy(np.random.default_rng(63).standard_normal((1, 1, 128))).bfloat16().to(cuda_device)
    v = good.clone()
    v[0, 0, 77] = value
    slot = np.array([blk * 16 + t])
    kvd.kvd_append_kv(c.pool.handle, 0, good, v, torch.from_numpy(slot).to(cuda_device))
    assert c.opool.append(good.float().cpu().numpy(), good.float().cpu().numpy(), slot) == 0
    ref, rlse, tol, ltol = c.reference()
    out, lse = run_many_rows(c)
    assert_within(out[:23], ref[:23], tol[:23], "earlier rows")
    assert_within(lse, rlse, ltol, "lse")
    assert not np.isfinite(out[23:, :, 77]).any()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "mixed", "int4"])
def test_many_rows_masked_slots_may_hold_anything(cuda_device, kind):
    c = Case(cuda_device, kind, 4, 1, [40], [300], seed=64, evict=0.2)
    bad = torch.full((1, 1, 128), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    for p in range(304):
        blk, t = int(c.bt[0, p // 16]), p % 16
        if p >= 300 or not (int(c.retain[blk]) >> t) & 1:
            x = bad if p % 2 else torch.full_like(bad, float("inf"))
            kvd.kvd_append_kv(c.pool.handle, 0, x, x, torch.tensor([blk * 16 + t], device=cuda_device))
    check_many_rows(c)
