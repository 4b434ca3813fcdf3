"""The latent cache on the GPU: append, read-back, absorbed and expanded attention against their formulas in 64 bits."""

import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from chunk_ref import rope_freqs_ref
from latent_ref import EPS, KEY, LAT, ROT, assert_within, attn_ref, prefill_ref, read_pool, slots_of, starts, tables

pytestmark = pytest.mark.gpu
BF16, FP8 = kvd.KVD_LATENT_BF16, kvd.KVD_LATENT_FP8
KINDS = pytest.mark.parametrize("kind", [BF16, FP8], ids=["bf16", "fp8"])
SCALE = 192 ** -0.5


def ok(pool):
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK


def oob(pool):
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_ERR_OOB


def rand(rng, *shape, factor=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * factor).bfloat16()


def to(dev, a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(dev)


def poisoned(layers, blocks, kind, dev):
    pool = kvd.LatentPool(layers, blocks, kind, device=dev)
    pool.mem.fill_(0xFF)   # NaN everywhere: unwritten slots must never leak
    return pool


# ------------------------------------------------------------------------ append
def turned(x, pos, rot, inter, rule):
    """fp64 rotation of x [n][..][64], and the sum of absolute products of each value."""
    theta, m = rope_freqs_ref(rot, 10000.0, **rule)
    ang = torch.from_numpy(pos.astype(np.float64)[:, None] * theta)
    ang = ang.view(len(pos), *[1] * (x.dim() - 2), rot // 2)
    c, s = m * ang.cos(), m * ang.sin()
    y, size = x.double().clone(), x.double().abs()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    xa, xb = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
    size[..., a] = size[..., b] = abs(m) * (xa.abs() + xb.abs())
    return y, size


def close_rotated(got, ref, size):
    # cos and sin are good to 2^-23 of 1 (and 2^-21 where the factor is applied), two products and a sum
    assert_within(got, ref, size * 2.0 ** -20, "rotated", torch.bfloat16)


@KINDS
@pytest.mark.parametrize("n,n_q,rot,inter,norm,fused", [
    (1, 1, 64, True, True, True), (1, 0, 64, True, False, False), (5, 3, 64, False, True, True), (70, 9, 62, False, False, True),
    (33, 4, 48, False, True, False), (40, 33, 30, True, True, True), (300, 128, 64, True, True, True), (17, 2, 2, False, False, False),
    (19, 5, 36, False, True, True)])
def test_append(cuda_device, kind, n, n_q, rot, inter, norm, fused):
    dev, rng = cuda_device, np.random.default_rng(n * 100 + rot)
    layers, nb = 2, n // 16 + 4
    pool = poisoned(layers, nb, kind, dev)
    before = pool.mem.clone()
    if fused:   # slices of one projection's output, and of all heads' queries
        x = rand(rng, n, KEY + 8, factor=3.0)
        lat, key = x[:, :LAT], x[:, LAT:KEY]
        q = rand(rng, n, max(n_q, 1), 192)[..., 128:]
        out = torch.full((n, max(n_q, 1), KEY), 9.0, dtype=torch.bfloat16)
    else:
        lat, key, q = rand(rng, n, LAT, factor=3.0), rand(rng, n, ROT), rand(rng, n, max(n_q, 1), ROT)
        out = torch.full((n, max(n_q, 1), KEY), 9.0, dtype=torch.bfloat16)
    w = (1.0 + 0.3 * rand(rng, LAT).float()).bfloat16() if norm else None
    pos = rng.integers(0, 1 << 24, n).astype(np.int32)
    slots = rng.permutation(nb * 16)[:n].astype(np.int64)
    skipped = rng.random(n) < 0.1 if n > 1 else np.zeros(1, bool)
    slots[skipped] = -1
    rule = dict(scaling="yarn", factor=8.0, original_len=4096, low=1.0, high=32.0) if rot == 64 and not norm else {}
    rope = kvd.Rope(rot, 10000.0, interleaved=inter, device=dev, **rule)
    xd = to(dev, x) if fused else None
    latd, keyd = (xd[:, :LAT], xd[:, LAT:KEY]) if fused else (to(dev, lat), to(dev, key))
    qd = to(dev, torch.cat([torch.zeros(n, q.shape[1], 128).bfloat16(), q], -1))[..., 128:]
    outd = to(dev, out)
    eps = 1e-5
    kvd.kvd_latent_append(pool.handle, 1, latd, keyd, to(dev, slots), positions=to(dev, pos), rope=rope,
                          norm_weight=None if w is None else to(dev, w), norm_eps=eps, q_rope=qd if n_q else None,
                          q_rope_out=outd[..., LAT:] if n_q else None)
    ok(pool)
    if n_q:
        close_rotated(outd[..., LAT:].cpu(), *turned(q, pos, rot, inter, rule))
        assert bool((outd[..., :LAT] == 9.0).all())
    values, codes, scales = read_pool(pool)
    y = lat.double()
    rel = 0.0
    if norm:   # 512 squares and their sum in fp32, a root, a quotient, two products
        y = y / (y.square().mean(1, keepdim=True) + eps).sqrt() * w.double()
        rel = 2.0 ** -18
    on = ~skipped
    r, size = turned(key, pos, rot, inter, rule)
    got = values[1][slots[on]]
    close_rotated(got[:, LAT:], r[on], size[on])
    if kind == BF16:
        assert_within(got[:, :LAT], y[on], y[on].abs() * rel, "latent", torch.bfloat16)
        if not norm:
            assert torch.equal(got[:, :LAT], y[on])
    else:
        s = y[on].abs().amax(1) / 448.0
        assert_within(scales[1].flatten()[slots[on]], s, s * (rel + 2.0 ** -23), "scale", torch.float32)
        # half a step of e4m3: 2^-4 of the value, 2^-10 scales below the smallest normal one
        assert_within(got[:, :LAT], y[on], y[on].abs() * (2.0 ** -4 + 2 * rel + 2.0 ** -22) + s[:, None] * 2.0 ** -10, "latent")
        assert float(codes[1].flatten(0, 0)[slots[on]].abs().amax(1).min()) == 448.0
    # nothing else is written: the other layer, the other slots
    after, was = (m.view(layers, nb, -1) for m in (pool.mem, before))
    assert torch.equal(after[0], was[0])
    fresh = kvd.LatentPool(layers, nb, kind, device=dev)
    fresh.mem.copy_(before)
    old = read_pool(fresh)[0][1]
    others = np.setdiff1d(np.arange(nb * 16), slots[on])
    assert bool(values[1][others].isnan().all()) and bool(old.isnan().all())


@KINDS
def test_append_without_rotation_or_norm_copies(cuda_device, kind):
    dev, rng = cuda_device, np.random.default_rng(3)
    pool = poisoned(1, 3, kind, dev)
    lat, key = rand(rng, 20, LAT), rand(rng, 20, ROT)
    lat[4] = 0.0                    # a zero row has scale 1
    key[5, 3], lat[6, 7] = float("inf"), float("nan")
    slots = np.arange(20, dtype=np.int64) + 3
    kvd.kvd_latent_append(pool.handle, 0, to(dev, lat), to(dev, key), to(dev, slots))
    ok(pool)
    values, codes, scales = read_pool(pool)
    got = values[0][slots]
    assert torch.equal(got[:, LAT:], key.double())
    if kind == BF16:
        assert torch.equal(got[:, :LAT].nan_to_num(7.0), lat.double().nan_to_num(7.0))
    else:
        assert float(scales[0].flatten()[slots[4]]) == 1.0 and bool((got[4, :LAT] == 0).all())
        assert bool(got[6, 7].isnan()) and int(got[6, :LAT].isnan().sum()) == 1


def test_append_of_rows_too_small_for_a_scale(cuda_device):
    """A row whose largest value over 448 is below fp32's smallest: scale 1 and zeros, not 0/0."""
    dev = cuda_device
    pool = poisoned(1, 1, FP8, dev)
    w = torch.zeros(LAT, dtype=torch.bfloat16)
    w[::2] = 2.0 ** -133
    ones = torch.ones(1, LAT, dtype=torch.bfloat16)   # y = w / sqrt(1 + 10^8): 2^-146 or 0
    kvd.kvd_latent_append(pool.handle, 0, to(dev, ones), to(dev, ones[:, :ROT].contiguous()), to(dev, np.zeros(1, np.int64)),
                          norm_weight=to(dev, w), norm_eps=1e8)
    ok(pool)
    values, _, scales = read_pool(pool)
    assert float(scales[0].flatten()[0]) == 1.0 and bool((values[0][0, :LAT] == 0).all())


@KINDS
def test_append_in_place_and_bad_tokens(cuda_device, kind):
    dev, rng, n = cuda_device, np.random.default_rng(4), 6
    pool = poisoned(1, 2, kind, dev)
    q = rand(rng, n, 5, 192)
    pos = np.array([0, 5, -1, 1 << 24, 7, 9], np.int32)
    slots = np.array([0, 1, 2, 3, 32, 1 << 40], np.int64)
    qd = to(dev, q)
    rope = kvd.Rope(64, 10000.0, device=dev)
    kvd.kvd_latent_append(pool.handle, 0, to(dev, rand(rng, n, LAT)), to(dev, rand(rng, n, ROT)), to(dev, slots),
                          positions=to(dev, pos), rope=rope, q_rope=qd[..., 128:])
    oob(pool)
    ref, size = turned(q[..., 128:], np.where((pos < 0) | (pos >= 1 << 24), 0, pos), 64, False, {})
    got = qd.cpu()
    assert torch.equal(got[..., :128], q[..., :128])
    good = [0, 1, 4, 5]
    close_rotated(got[good][..., 128:], ref[good], size[good])
    assert torch.equal(got[2:4], q[2:4])                      # skipped whole
    values = read_pool(pool)[0][0]
    assert bool(values[:2].isfinite().all()) and bool(values[2:].isnan().all())


# ------------------------------------------------------------------------ gather
class Cache:
    """A pool with random rows of requests in shuffled blocks, everything else NaN."""

    def __init__(self, dev, kind, lens, seed=0, spare=3, layers=1, factor=1.0):
        rng = np.random.default_rng(seed)
        self.dev, self.kind, self.lens = dev, kind, list(lens)
        self.bt, self.nb = tables(lens, spare, seed)
        self.pool = poisoned(layers, self.nb, kind, dev)
        self.layer = layers - 1
        for b, n in enumerate(lens):
            if n > 0:
                self.put(b, 0, n, rand(rng, n, LAT, factor=factor), rand(rng, n, ROT, factor=factor))
        self.rng = rng

    def put(self, b, lo, hi, lat, key):
        kvd.kvd_latent_append(self.pool.handle, self.layer, to(self.dev, lat), to(self.dev, key),
                              to(self.dev, slots_of(self.bt, b, lo, hi)))

    def rows(self):
        return read_pool(self.pool)[0][self.layer]


@KINDS
@pytest.mark.parametrize("first,counts", [((0,), (1,)), ((3,), (40,)), ((0, 15, 31, 7), (17, 0, 2, 100))])
@pytest.mark.parametrize("stride", [576, 640])
def test_gather(cuda_device, kind, first, counts, stride):
    dev = cuda_device
    c = Cache(dev, kind, [a + n for a, n in zip(first, counts)], seed=5, layers=2)
    start = starts(counts) + 2
    out = torch.full((int(start[-1]) + 3, stride), 9.0, dtype=torch.bfloat16, device=dev)
    kvd.kvd_latent_gather(c.pool.handle, 1, to(dev, c.bt), to(dev, start), out[:, :KEY],
                          first=to(dev, np.array(first, np.int32)))
    ok(c.pool)
    values, codes, scales = read_pool(c.pool)
    want = torch.full((out.shape[0], KEY), 9.0, dtype=torch.bfloat16)
    for b, n in enumerate(counts):
        if n:
            at = slots_of(c.bt, b, first[b], first[b] + n)
            v = values[1][at].float()
            if kind == FP8:    # the product in fp32, rounded once
                v[:, :LAT] = codes[1].flatten(0, 0)[at].float() * scales[1].flatten()[at].float()[:, None]
            want[start[b]:start[b + 1]] = v.bfloat16()
    assert torch.equal(out[:, :KEY].cpu(), want)
    assert bool((out[:, KEY:] == 9.0).all())


@KINDS
def test_gather_skips_what_is_wrong(cuda_device, kind):
    dev = cuda_device
    c = Cache(dev, kind, [40, 40, 40], seed=6)
    bt = c.bt.copy()
    bt[1, 1] = c.nb                    # outside the pool: its 16 rows are left
    for start, first, skipped in (([0, 40, 80, 120], [0, 0, 9], [2]), ([0, 40, 30, 121], [0, 0, 0], [1, 2]),
                                  ([0, 40, 80, 120], [-1, 0, 0], [0])):
        out = torch.full((120, KEY), 9.0, dtype=torch.bfloat16, device=dev)
        kvd.kvd_latent_gather(c.pool.handle, 0, to(dev, bt), to(dev, np.array(start, np.int32)), out,
                              first=to(dev, np.array(first, np.int32)))
        oob(c.pool)
        rows = c.rows()
        for b in range(3):
            if b in skipped:
                continue
            got = out[start[b]:start[b] + 40].cpu()
            at = slots_of(c.bt, b, 0, 40)
            keep = np.ones(40, bool)
            if b == 1:
                keep[16:32] = False
                assert bool((got[16:32] == 9.0).all())
            assert torch.equal(got[keep], rows[at][keep].float().bfloat16())


def test_gather_of_pairs_that_overlap(cuda_device):
    """Every second pair is the whole of out, the others are backwards: 2^31 chunks of eight rows, more than 32 bits count."""
    dev, rng, batch, n = cuda_device, np.random.default_rng(7), 2048, 1 << 24
    pool = poisoned(1, 1, BF16, dev)
    rows = rand(rng, 16, KEY)
    kvd.kvd_latent_append(pool.handle, 0, to(dev, rows[:, :LAT]), to(dev, rows[:, LAT:]), to(dev, np.arange(16, dtype=np.int64)))
    table = torch.zeros(batch, n // 16, dtype=torch.int32, device=dev)
    start = torch.tensor([0, n] * (batch // 2) + [0], dtype=torch.int32, device=dev)
    out = torch.full((n, KEY), 9.0, dtype=torch.bfloat16, device=dev)
    kvd.kvd_latent_gather(pool.handle, 0, table, start, out)
    oob(pool)
    want = to(dev, rows).repeat(1 << 12, 1)
    assert all(torch.equal(x, want) for x in out.split(1 << 16))


# ------------------------------------------------------------- absorbed attention
class Attn(Cache):
    def __init__(self, dev, kind, n_q, q_lens, lens, seed=0, evict=0.0, **kw):
        super().__init__(dev, kind, lens, seed, **kw)
        self.n_q = n_q
        self.start = starts(q_lens)
        self.q = rand(self.rng, int(self.start[-1]), n_q, KEY)
        self.retain = None
        if evict:
            keep = self.rng.random((self.nb, 16)) >= evict
            self.retain = (keep << np.arange(16)).sum(1).astype(np.uint16)

    def args(self):
        dev = self.dev
        return dict(q=to(dev, self.q), q_start=to(dev, self.start), block_table=to(dev, self.bt),
                    seq_lens=to(dev, np.array(self.lens, np.int32)),
                    retain_mask=None if self.retain is None else to(dev, self.retain.view(np.int16)),
                    workspace=torch.empty(kvd.kvd_latent_workspace_bytes(self.pool.handle, self.n_q, len(self.lens)),
                                          dtype=torch.uint8, device=dev).fill_(0xFF))

    def run(self, dtype=torch.float32, scale=None, a=None, **kw):
        a = a or self.args()
        out = torch.full((*self.q.shape[:2], LAT), 9.0, dtype=dtype, device=self.dev)
        lse = torch.full(self.q.shape[:2], 9.0, dtype=torch.float32, device=self.dev)
        kvd.kvd_latent_attn(self.pool.handle, self.layer, out=out, lse_out=lse, softmax_scale=scale, **{**a, **kw})
        return out, lse

    def check(self, dtype=torch.float32, scale=None, device="cpu", absent=(), rows=None):
        out, lse = self.run(dtype, scale)
        ref, rl, tol, lt = attn_ref(self.rows() if rows is None else rows, self.q, self.start, self.bt, self.lens, self.retain,
                                    SCALE if scale is None else scale, device, absent)
        assert_within(lse, rl, lt, "lse")
        assert_within(out, ref, tol, "out", dtype)


SHAPES = [(1, [1], [1]), (16, [1, 1], [17, 1]), (5, [3, 0, 70], [3, 20, 333]), (64, [2], [130]), (65, [2, 1], [100, 64]),
          (128, [1, 2], [129, 700]), (20, [7], [64]), (256, [1], [65]), (33, [5, 1, 1], [63, 64, 65]), (7, [64], [64]),
          (3, [40, 1], [41, 1000])]


@KINDS
@pytest.mark.parametrize("n_q,q_lens,lens", SHAPES)
@pytest.mark.parametrize("evict", [0.0, 0.3])
def test_attn(cuda_device, kind, n_q, q_lens, lens, evict):
    c = Attn(cuda_device, kind, n_q, q_lens, lens, seed=n_q, evict=evict)
    c.check()
    c.check(torch.bfloat16)
    ok(c.pool)


@KINDS
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 2.0])
def test_attn_scales(cuda_device, kind, scale):
    c = Attn(cuda_device, kind, 9, [3, 1], [75, 200], seed=2, evict=0.2)
    c.check(scale=scale)


@KINDS
def test_attn_long_rows_are_cut_and_joined(cuda_device, kind):
    """A few long contexts over every multiprocessor: parts of one unit in many CTAs, several units in one."""
    for n_q, q_lens, lens in ((16, [1], [20011]), (128, [1, 3], [5000, 9001]), (40, [1] * 40, list(range(200, 1000, 20))),
                              (8, [100], [4000])):
        c = Attn(cuda_device, kind, n_q, q_lens, lens, seed=8, evict=0.1)
        c.check(torch.bfloat16, device=cuda_device)
        c.check(device=cuda_device)
        ok(c.pool)


@KINDS
@pytest.mark.parametrize("n_q,q_lens,lens", [
    (64, [1] * 12, [4096] * 12), (40, [1] * 9, [5000, 37, 2300, 1, 0, 4100, 3000, 5001, 64]), (128, [1] * 3, [2500, 40, 3000]),
    (16, [1] * 4, [4000] * 4), (5, [2, 2, 0, 1], [3000, 2, 0, 2999]), (70, [3] * 4, [2100] * 4), (1, [1] * 32, [1500] * 32)])
def test_attn_cut_units(cuda_device, kind, n_q, q_lens, lens):
    """Few requests, whose units get whole shares, and cut ones: joins of few and of many parts, of few and of many rows."""
    q_lens = [q if n else 0 for q, n in zip(q_lens, lens)]
    c = Attn(cuda_device, kind, n_q, q_lens, lens, seed=n_q + len(lens), evict=0.05)
    c.check(torch.bfloat16, device=cuda_device)
    c.check(device=cuda_device)
    ok(c.pool)


@KINDS
@pytest.mark.parametrize("n", [1, 70, 5000])
def test_attn_of_one_token_is_its_value(cuda_device, kind, n):
    """Where a row's whole weight is on one token, that weight's rounding (in 8 bits with the token's scale) cancels."""
    dev, rng = cuda_device, np.random.default_rng(n)
    c = Cache(dev, kind, [n], seed=n)
    at = rng.integers(0, n, 16)
    key = torch.zeros(n, ROT, dtype=torch.bfloat16)
    q = torch.zeros(1, 16, KEY, dtype=torch.bfloat16)
    for h, j in enumerate(at):   # two of the rotated dims tell a head's token: a logit of 2^16·scale, others at most half of it
        key[j, h] = key[j, 16 + h] = 256.0
        q[0, h, LAT + h] = q[0, h, LAT + 16 + h] = 128.0
    lat = rand(rng, n, LAT)
    c.put(0, 0, n, lat, key)
    out, lse = torch.zeros(1, 16, LAT, device=dev), torch.zeros(1, 16, device=dev)
    ws = torch.empty(kvd.kvd_latent_workspace_bytes(c.pool.handle, 16, 1), dtype=torch.uint8, device=dev)
    kvd.kvd_latent_attn(c.pool.handle, 0, to(dev, q), to(dev, np.array([0, 1], np.int32)), to(dev, c.bt), to(dev, np.array([n], np.int32)),
                        ws, out, softmax_scale=SCALE, lse_out=lse)
    ok(c.pool)
    want = c.rows()[slots_of(c.bt, 0, 0, n)][at, :LAT]
    # a quotient, two products and at most 147 parts' sums of which one is not 0
    assert_within(out[0], want, want.abs() * 2.0 ** -21, "out")
    assert_within(lse[0], torch.full((16,), 2.0 ** 16 * SCALE, dtype=torch.float64), torch.full((16,), 2.0 ** 16 * SCALE * 2.0 ** -21, dtype=torch.float64), "lse")


@KINDS
def test_attn_growing_logits_move_the_reference(cuda_device, kind):
    """Each tile's maximum passes the last one's by more than the lazy border, so O is rescaled many times."""
    dev, n = cuda_device, 900
    c = Attn(dev, kind, 4, [2], [n], seed=9)
    rng = np.random.default_rng(1)
    q = torch.zeros(2, 4, KEY).bfloat16()
    q[..., LAT] = 1.0
    c.q = q
    key = torch.zeros(n, ROT).bfloat16()
    key[:, 0] = torch.arange(n).float().bfloat16()
    c.put(0, 0, n, rand(rng, n, LAT), key)
    c.check(scale=0.5)
    c.check(scale=-0.5)


@KINDS
def test_attn_nothing_retained(cuda_device, kind):
    dev = cuda_device
    c = Attn(dev, kind, 6, [2, 1], [40, 3000], seed=3)
    c.retain = np.zeros(c.nb, np.uint16)
    out, lse = c.run()
    assert bool((out == 0).all()) and bool((lse == -torch.inf).all())
    c.retain[c.bt[0, 0]] = 1 << 5      # one position of the first request
    c.check()
    ok(c.pool)


@KINDS
def test_attn_rows_outside_every_request_are_left(cuda_device, kind):
    c = Attn(cuda_device, kind, 6, [3, 2], [40, 30], seed=3)
    c.q = torch.cat([c.q, torch.full((4, 6, KEY), float("nan")).bfloat16()])
    out, lse = c.run()
    ref, rl, tol, lt = attn_ref(c.rows(), c.q, c.start, c.bt, c.lens, None, SCALE)
    assert_within(out[:5], ref[:5], tol[:5], "out")
    assert bool((out[5:] == 9.0).all()) and bool((lse[5:] == 9.0).all())


@KINDS
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n_q,T,N", [(8, 8, 100), (8, 8, 3000), (20, 70, 70), (128, 2, 400)])
def test_attn_later_tokens_do_not_reach_earlier_rows(cuda_device, kind, bad, n_q, T, N):
    """A new token that is not finite: the rows before it do not notice, the others have what the formula gives."""
    dev = cuda_device
    c = Attn(dev, kind, n_q, [T], [N], seed=12)
    clean, clean_lse = c.run()
    j = T // 2 + 1 if T > 2 else 1
    lat, key = rand(c.rng, 1, LAT), rand(c.rng, 1, ROT)
    lat[0, 100] = bad
    pos = N - T + j
    c.put(0, pos, pos + 1, lat, key)
    out, lse = c.run()
    ref, rl, tol, lt = attn_ref(c.rows(), c.q, c.start, c.bt, [N], None, SCALE, dev)
    assert bool(out[:j].isfinite().all()) and bool(lse[:j].isfinite().all())
    assert_within(out[:j], ref[:j], tol[:j], "rows before it")
    assert_within(lse[:j], rl[:j], lt[:j], "lse before it")
    assert torch.equal(out[j:].isnan().cpu(), ref[j:].isnan().cpu()) or math.isinf(bad)
    if math.isnan(bad):
        assert bool(out[j:].isnan().any(-1).all())


@KINDS
def test_attn_masked_slots_may_hold_anything(cuda_device, kind):
    dev = cuda_device
    c = Attn(dev, kind, 12, [2, 1], [100, 700], seed=13, evict=0.4)
    want = c.run()
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        for b, n in enumerate(c.lens):
            lat, key = torch.full((1, LAT), bad).bfloat16(), torch.full((1, ROT), bad).bfloat16()
            for pos in range(n):
                if not c.retain[c.bt[b, pos // 16]] >> (pos % 16) & 1 and pos % 3 == 0:
                    c.put(b, pos, pos + 1, lat, key)
        got = c.run()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@KINDS
def test_attn_non_finite_tokens_that_are_attended(cuda_device, kind):
    dev = cuda_device
    c = Attn(dev, kind, 4, [1], [90], seed=14)
    lat = torch.zeros(1, LAT).bfloat16()
    lat[0, 5] = float("nan")
    c.put(0, 50, 51, lat, torch.zeros(1, ROT).bfloat16())
    out, lse = c.run()
    assert bool(out[..., 5].isnan().all()) and bool(lse.isnan().all())


@KINDS
def test_attn_wrong_lengths_and_blocks(cuda_device, kind):
    dev = cuda_device
    c = Attn(dev, kind, 6, [3, 2, 4], [40, 30, 100], seed=15)
    rows = c.rows()
    for lens in ([2, 30, 100], [40, 16 * c.bt.shape[1] + 1, 100], [40, 30, -5]):
        a = c.args()
        a["seq_lens"] = to(dev, np.array(lens, np.int32))
        out, lse = c.run(a=a)
        oob(c.pool)
        good = [n == m for n, m in zip(lens, c.lens)]
        ref, rl, tol, lt = attn_ref(rows, c.q, c.start, c.bt, [n if g else 0 for n, g in zip(lens, good)], None, SCALE)
        for b, g in enumerate(good):
            r = slice(c.start[b], c.start[b + 1])
            if g:
                assert_within(out[r], ref[r], tol[r], "out")
            else:
                assert bool((out[r] == 0).all()) and bool((lse[r] == -torch.inf).all())
    for start, skipped in (([0, 3, 2, 9], [1]), ([0, 3, 5, 10], [2]), ([-1, 3, 5, 9], [0])):
        a = c.args()
        a["q_start"] = to(dev, np.array(start, np.int32))
        out, lse = c.run(a=a)
        oob(c.pool)
        for b in skipped:
            if start[b] >= 0 and b == 2:
                assert bool((out[start[b]:] == 9.0).all())
    for bad in (-1, c.nb, 1 << 30):
        bt = c.bt.copy()
        bt[2, 1] = bad
        a = c.args()
        a["block_table"] = to(dev, bt)
        out, lse = c.run(a=a)
        oob(c.pool)
        ref, rl, tol, lt = attn_ref(rows, c.q, c.start, bt, c.lens, None, SCALE, absent=[bad])
        assert_within(out, ref, tol, "out")


@KINDS
def test_attn_starts_that_break(cuda_device, kind):
    """A pair of q_start that runs backwards, or out of q: that request's rows are left, the others' are as they should be."""
    dev = cuda_device
    c = Attn(dev, kind, 6, [3, 2, 4], [40, 30, 100], seed=15)
    rows = c.rows()
    for start, good in (([0, 3, 2, 9], [0, 2]), ([0, 3, 5, 10], [0, 1]), ([-1, 3, 5, 9], [1, 2]), ([0, 10, 5, 9], [2]), ([3, 3, 3, 9], [2])):
        a = c.args()
        a["q_start"] = to(dev, np.array(start, np.int32))
        out, lse = c.run(a=a)
        if start[0] != 3:
            oob(c.pool)
        owners = np.zeros(9, int)
        for b in good:
            owners[start[b]:start[b + 1]] += 1
        for b in good:
            lens = [n if i == b else 0 for i, n in enumerate(c.lens)]
            ref, rl, tol, lt = attn_ref(rows, c.q, start, c.bt, lens, None, SCALE)
            mine = [r for r in range(start[b], start[b + 1]) if owners[r] == 1]   # (where two overlap it is either's)
            assert_within(out[mine], ref[mine], tol[mine], "out")
            assert_within(lse[mine], rl[mine], lt[mine], "lse")
        assert bool((out[owners == 0] == 9.0).all()) and bool((lse[owners == 0] == 9.0).all())


@KINDS
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("n_q,T,N", [(8, 8, 100), (8, 8, 3000), (20, 70, 70), (128, 2, 400)])
def test_attn_of_an_infinite_token(cuda_device, kind, bad, n_q, T, N):
    """One value of a new token's latent is infinite.  A head that gives it the logit +inf has no finite value; one that gives it
    -inf has the others' softmax, and in that dim 0·inf.  In 8 bits the token's scale is infinite and its codes times it NaN."""
    dev, j = cuda_device, T // 2
    c = Attn(dev, kind, n_q, [T], [N], seed=22)
    pos = N - T + j
    lat, key = rand(c.rng, 1, LAT), rand(c.rng, 1, ROT)
    lat[0, 100] = bad
    c.retain = np.full(c.nb, 0xFFFF, np.uint16)
    c.put(0, pos, pos + 1, lat, key)
    out, lse = c.run()
    rows = c.rows()
    c.retain[c.bt[0, pos // 16]] ^= 1 << (pos % 16)   # the others' softmax
    ref, rl, tol, lt = attn_ref(rows, c.q, c.start, c.bt, c.lens, c.retain, SCALE, dev)
    assert_within(out[:j], ref[:j], tol[:j], "rows before it")
    assert_within(lse[:j], rl[:j], lt[:j], "lse before it")
    out, lse, ref, rl, tol, lt = (x[j:].cpu() for x in (out, lse, ref, rl, tol, lt))
    if kind == FP8:
        assert bool(out.isnan().all()) and bool(lse.isnan().all())
        return
    most = c.q[j:, :, 100].float() * bad > 0
    assert bool(out[most].isnan().all()) and not bool(lse[most].isfinite().any())
    assert bool(out[~most][:, 100].isnan().all())
    rest = np.arange(LAT) != 100
    assert_within(out[~most][:, rest], ref[~most][:, rest], tol[~most][:, rest], "the others")
    assert_within(lse[~most], rl[~most], lt[~most], "lse")


@KINDS
def test_attn_same_bits_streams_and_graphs(cuda_device, kind):
    dev = cuda_device
    c = Attn(dev, kind, 16, [1, 3, 1], [3000, 500, 77], seed=16, evict=0.1)
    d = Attn(dev, kind, 128, [2, 1], [900, 2500], seed=17)
    want, dwant = c.run(torch.bfloat16), d.run(torch.bfloat16)
    assert all(torch.equal(x, y) for x, y in zip(c.run(torch.bfloat16), want))
    # two calls at once, each with its workspace
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = c.args(), d.args()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            x = c.run(torch.bfloat16, a=a)
        with torch.cuda.stream(s2):
            y = d.run(torch.bfloat16, a=b)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(x, want)) and all(torch.equal(p, q) for p, q in zip(y, dwant))
    # captured, replayed over new contents
    out = torch.zeros((*c.q.shape[:2], LAT), dtype=torch.bfloat16, device=dev)
    lse = torch.zeros(c.q.shape[:2], dtype=torch.float32, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvd.kvd_latent_attn(c.pool.handle, c.layer, out=out, lse_out=lse, **a)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    a["seq_lens"].copy_(to(dev, np.array([2000, 400, 50], np.int32)))
    g.replay()
    torch.cuda.synchronize()
    c.lens = [2000, 400, 50]
    ref, rl, tol, lt = attn_ref(c.rows(), c.q, c.start, c.bt, c.lens, c.retain, SCALE)
    assert_within(out, ref, tol, "out", torch.bfloat16)
    assert_within(lse, rl, lt, "lse")
    ok(c.pool)


def test_attn_repairs_long_rows_in_peace(cuda_device):
    """A NaN in the last token, 120,000 positions, whole units: the first token's rows are computed again for longer than
    the other warps' waits last."""
    dev, sms, blocks, n_q = cuda_device, torch.cuda.get_device_properties(0).multi_processor_count, 7500, 32
    B, N = 2 * sms, 16 * blocks
    pool = poisoned(1, 2, BF16, dev)
    rng = np.random.default_rng(9)
    lat, key = rand(rng, 32, LAT), rand(rng, 32, ROT)
    lat[31, 5] = float("nan")
    kvd.kvd_latent_append(pool.handle, 0, to(dev, lat), to(dev, key), to(dev, np.arange(32, dtype=np.int64)))
    table = torch.zeros(B, blocks, dtype=torch.int32, device=dev)
    table[:, -1] = 1
    q = torch.zeros(2 * B, n_q, KEY, dtype=torch.bfloat16, device=dev)
    out, lse = torch.zeros(2 * B, n_q, LAT, device=dev), torch.zeros(2 * B, n_q, device=dev)
    ws = torch.empty(kvd.kvd_latent_workspace_bytes(pool.handle, n_q, B), dtype=torch.uint8, device=dev)
    kvd.kvd_latent_attn(pool.handle, 0, q, torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device=dev), table,
                        torch.full((B,), N, dtype=torch.int32, device=dev), ws, out, softmax_scale=SCALE, lse_out=lse)
    ok(pool)
    # every weight is 1; N additions in a row, each off by at most 2^-24 of a sum of absolute values
    x = lat[:31].double()
    mean, size = ((blocks - 1) * y[:16].sum(0) / (N - 1) + y[16:].sum(0) / (N - 1) for y in (x, x.abs()))
    assert_within(out[::2].cpu(), mean.expand(B, n_q, LAT), (2 * N * 2.0 ** -24 * size).expand(B, n_q, LAT), "out")
    assert float((lse[::2].double() - np.log(N - 1)).abs().max()) < 2 * N * 2.0 ** -24
    assert bool(out[1::2, :, 5].isnan().all())


def test_attn_of_the_longest_request(cuda_device):
    """2^31 − 1 positions, all in one block: lengths and tiles stay within their types."""
    dev, rng = cuda_device, np.random.default_rng(8)
    pool = poisoned(1, 1, BF16, dev)
    lat = torch.ones(16, LAT, dtype=torch.bfloat16)
    kvd.kvd_latent_append(pool.handle, 0, to(dev, lat), to(dev, rand(rng, 16, ROT)), to(dev, np.arange(16, dtype=np.int64)))
    table = torch.zeros(1, 1 << 27, dtype=torch.int32, device=dev)
    q = torch.zeros(1, 1, KEY, dtype=torch.bfloat16, device=dev)
    out, lse = torch.zeros(1, 1, LAT, device=dev), torch.zeros(1, 1, device=dev)
    ws = torch.empty(kvd.kvd_latent_workspace_bytes(pool.handle, 1, 1), dtype=torch.uint8, device=dev)
    kvd.kvd_latent_attn(pool.handle, 0, q, torch.tensor([0, 1], dtype=torch.int32, device=dev), table,
                        torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=dev), ws, out, softmax_scale=SCALE, lse_out=lse)
    ok(pool)
    # every weight is 1; a CTA's sum takes 2^25/152 tiles of 16 additions a lane, each off by at most 2^-24 of the sum
    slack = (2 ** 25 // 152 + 1) * 16 * 2.0 ** -24
    assert abs(float(lse) - 31 * np.log(2.0)) < -np.log1p(-slack)
    assert bool(((out - 1).abs() < 2 * slack).all())


def test_attn_many_requests(cuda_device):
    rng = np.random.default_rng(18)
    q_lens = rng.integers(0, 3, 2048).tolist()
    lens = [t + int(n) for t, n in zip(q_lens, rng.integers(0, 60, 2048))]
    c = Attn(cuda_device, BF16, 4, q_lens, lens, seed=18)
    c.check(device=cuda_device)
    ok(c.pool)


def test_attn_shared_blocks(cuda_device):
    """Two requests with one prefix: the same blocks in both rows of the table."""
    c = Attn(cuda_device, BF16, 10, [1, 2], [200, 180], seed=19)
    c.bt[1, :5] = c.bt[0, :5]
    c.check()


# ------------------------------------------------------------- expanded attention
class Prefill:
    def __init__(self, dev, n_q, q_lens, kv_lens, seed=0, sliced=True, before=0, behind=0):
        rng = np.random.default_rng(seed)
        self.dev, self.n_q = dev, n_q
        self.start, self.kv_start = starts(q_lens) + before, starts(kv_lens) + before
        n, m = int(self.start[-1]) + behind, int(self.kv_start[-1]) + behind
        self.q = rand(rng, n, n_q, 192)
        kv = rand(rng, m, n_q, 256)
        self.k, self.v, self.r = kv[..., :128], kv[..., 128:], rand(rng, m, KEY)[:, LAT:]
        self.sliced = sliced

    def run(self, causal=True, dtype=torch.float32, scale=None, pool=None):
        dev = self.dev
        self.pool = pool or kvd.LatentPool(1, 1, device=dev)
        if self.sliced:
            kv = to(dev, torch.cat([self.k, self.v], -1))
            k, v = kv[..., :128], kv[..., 128:]
            r = to(dev, torch.cat([torch.zeros(self.r.shape[0], LAT).bfloat16(), self.r], -1))[:, LAT:]
        else:
            k, v, r = to(dev, self.k.contiguous()), to(dev, self.v.contiguous()), to(dev, self.r.contiguous())
        out = torch.full((*self.q.shape[:2], 128), 9.0, dtype=dtype, device=dev)
        lse = torch.full(self.q.shape[:2], 9.0, dtype=torch.float32, device=dev)
        kvd.kvd_latent_prefill(self.pool.handle, to(dev, self.q), to(dev, self.start), k, v, r, to(dev, self.kv_start), out,
                               causal=causal, softmax_scale=scale, lse_out=lse)
        return out, lse

    def ref(self, causal=True, scale=None):
        return prefill_ref(self.q, self.k, self.v, self.r, self.start, self.kv_start, causal, SCALE if scale is None else scale,
                           self.dev)

    def check(self, causal=True, dtype=torch.float32, scale=None):
        out, lse = self.run(causal, dtype, scale)
        ok(self.pool)
        ref, rl, tol, lt = self.ref(causal, scale)
        rows = np.concatenate([np.arange(a, b) for a, b in zip(self.start[:-1], self.start[1:])]).astype(np.int64)
        assert_within(lse[rows], rl[rows], lt[rows], "lse")
        assert_within(out[rows], ref[rows], tol[rows], "out", dtype)
        outside = np.setdiff1d(np.arange(self.q.shape[0]), rows)
        assert bool((out[outside] == 9.0).all()) and bool((lse[outside] == 9.0).all())


@pytest.mark.parametrize("n_q,q_lens,kv_lens", [
    (1, [1], [1]), (3, [5, 0, 200], [9, 4, 200]), (2, [129], [129]), (2, [128], [300]), (1, [256], [256]), (1, [257], [700]),
    (5, [1, 1], [1000, 127]), (4, [30], [10]), (3, [7, 4], [0, 4]), (2, [300, 300], [200, 1]), (8, [64, 600], [64, 640])])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill(cuda_device, n_q, q_lens, kv_lens, causal):
    c = Prefill(cuda_device, n_q, q_lens, kv_lens, seed=n_q, sliced=n_q % 2 == 1, before=n_q, behind=3)
    c.check(causal)
    c.check(causal, torch.bfloat16)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 2.0])
def test_prefill_scales(cuda_device, scale):
    Prefill(cuda_device, 3, [140, 3], [150, 300], seed=2).check(scale=scale)


def test_prefill_of_many_units(cuda_device):
    """More units than multiprocessors: every CTA takes several, some of them empty halves."""
    Prefill(cuda_device, 40, [1, 300, 129, 17, 512, 0, 100], [500, 300, 130, 1000, 512, 3, 900], seed=3).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_out_on_any_16_bytes(cuda_device, dtype):
    c = Prefill(cuda_device, 3, [140], [150], seed=12)
    want, _ = c.run(dtype=dtype)
    buf = torch.full((want.numel() + 16,), 9.0, dtype=dtype, device=cuda_device)
    at = 16 // want.element_size()
    out = buf[at:at + want.numel()].view(want.shape)
    k, v, r = (to(cuda_device, x.contiguous()) for x in (c.k, c.v, c.r))
    kvd.kvd_latent_prefill(c.pool.handle, to(cuda_device, c.q), to(cuda_device, c.start), k, v, r, to(cuda_device, c.kv_start), out)
    assert out.data_ptr() % 32 == 16 and torch.equal(out, want)
    assert bool((buf[:at] == 9.0).all()) and bool((buf[at + want.numel():] == 9.0).all())


def test_prefill_of_more_blocks_than_are_sorted(cuda_device):
    """More than 512 blocks of 256 tokens: they are taken as they come."""
    rng = np.random.default_rng(13)
    q = rng.integers(1, 300, 600)
    Prefill(cuda_device, 1, q.tolist(), (q + rng.integers(0, 9, 600)).tolist(), seed=13).check()


def test_prefill_many_requests(cuda_device):
    rng = np.random.default_rng(4)
    q = rng.integers(0, 4, 2048)
    Prefill(cuda_device, 2, q.tolist(), (q + rng.integers(0, 9, 2048)).tolist(), seed=4).check()


def test_prefill_without_keys(cuda_device):
    c = Prefill(cuda_device, 2, [3, 200], [0, 0], seed=5)
    for causal in (True, False):
        out, lse = c.run(causal)
        assert bool((out == 0).all()) and bool((lse == -torch.inf).all())


def test_prefill_growing_logits_move_the_reference(cuda_device):
    c = Prefill(cuda_device, 2, [10], [900], seed=6)
    c.q.zero_()
    c.q[..., 128] = 1.0
    c.r[:, 0] = torch.arange(900).float().bfloat16()
    c.check(scale=0.5)
    c.check(scale=-0.5, causal=False)


@pytest.mark.parametrize("n_q,q_lens,kv_lens", [
    (3, [100, 300, 1], [900, 1000, 5000]), (40, [33] * 6, [2000] * 6), (40, [128, 129, 384, 20], [640, 640, 900, 3000]),
    (1, [128], [513]), (2, [60], [511]), (1, [1], [385]), (32, [1, 2] * 10, [600, 1300] * 10), (9, [390, 64, 700, 5] * 5, [390, 777, 5000, 640] * 5)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_few_rows_behind_many_keys(cuda_device, n_q, q_lens, kv_lens, causal):
    """Rows of one warpgroup alone, over several tiles of keys."""
    c = Prefill(cuda_device, n_q, q_lens, kv_lens, seed=n_q + 1)
    c.check(causal)
    c.check(causal, torch.bfloat16)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,N,j", [(100, 700, 60), (60, 513, 1), (128, 1000, 127)])
def test_prefill_later_tokens_behind_many_keys(cuda_device, bad, T, N, j):
    test_prefill_later_tokens_do_not_reach_earlier_rows(cuda_device, bad, T, N, j)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,N,j", [(100, 100, 50), (300, 400, 150), (300, 300, 299), (2, 130, 1)])
def test_prefill_later_tokens_do_not_reach_earlier_rows(cuda_device, bad, T, N, j):
    c = Prefill(cuda_device, 3, [T], [N], seed=7)
    c.v[N - T + j, 1, 9] = bad
    c.k[N - T + j, 2, 9] = bad
    out, lse = c.run()
    ref, rl, tol, lt = c.ref()
    assert_within(out[:j], ref[:j], tol[:j], "rows before it")
    assert_within(lse[:j], rl[:j], lt[:j], "lse before it")
    assert_within(out[:, 0], ref[:, 0], tol[:, 0], "the other head")
    assert_within(out[:, 1, :9], ref[:, 1, :9], tol[:, 1, :9], "the other dims")
    if math.isnan(bad):
        assert bool(out[j:, 1, 9].isnan().all()) and bool(out[j:, 2].isnan().all())
    else:
        assert bool((out[j:, 1, 9] == bad).all())


def test_prefill_repairs_long_rows_in_peace(cuda_device):
    """A NaN in the last of 131,072 keys, 65 rows: those before it are computed again, 32 a warp, for longer than the other
    warps' waits last."""
    dev, rng, T, N = cuda_device, np.random.default_rng(10), 65, 1 << 17
    pool = kvd.LatentPool(1, 1, BF16, device=dev)
    v = rand(rng, 64, 128).repeat(N // 64, 1).view(N, 1, 128)
    v[-1, 0, 3] = float("nan")
    zeros = torch.zeros(N, 1, 192, dtype=torch.bfloat16, device=dev)
    out, lse = torch.zeros(T, 1, 128, device=dev), torch.zeros(T, 1, device=dev)
    starts = [torch.tensor([0, n], dtype=torch.int32, device=dev) for n in (T, N)]
    kvd.kvd_latent_prefill(pool.handle, zeros[:T], starts[0], zeros[..., :128], to(dev, v), zeros[:, 0, 128:], starts[1], out, lse_out=lse)
    ok(pool)
    # every weight is 1; N additions in a row, each off by at most 2^-24 of a sum of absolute values
    ends = torch.arange(N - T + 1, N)[:, None]
    x = v[:, 0].double().nan_to_num(0.0)
    mean, size = (y.cumsum(0)[ends[:, 0] - 1] / ends for y in (x, x.abs()))
    assert_within(out[:-1, 0].cpu(), mean, 2 * N * 2.0 ** -24 * size, "out")
    assert float((lse[:-1, 0].cpu().double() - ends[:, 0].double().log()).abs().max()) < 2 * N * 2.0 ** -24
    assert bool(out[-1, 0, 3].isnan())


def test_prefill_what_no_row_attends_may_be_anything(cuda_device):
    """Rows between and behind the requests, and the keys behind a request's last."""
    c = Prefill(cuda_device, 3, [50, 20], [70, 33], seed=8, before=4, behind=200)
    want = c.run()
    for x in (c.q, c.k, c.v, c.r):
        x[:4], x[-200:] = float("nan"), float("inf")
    got = c.run()
    rows = slice(4, 74)
    assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][rows], want[1][rows])
    one, d = Prefill(cuda_device, 3, [50, 20], [70, 33], seed=8, before=4, behind=200), c
    one.v[74:], one.r[74:] = float("nan"), float("nan")       # the other request's keys
    got = one.run()
    assert torch.equal(got[0][4:54], want[0][4:54])
    assert d.n_q == 3


@pytest.mark.parametrize("n_q,T,N,causal", [
    (5, 200, 250, True), (5, 254, 383, True), (40, 130, 380, True), (2, 129, 1000, True), (3, 456, 600, True),
    (5, 200, 300, False), (3, 256, 10, False), (40, 255, 129, False), (2, 600, 383, False), (1, 129, 1, False)])
def test_prefill_keys_of_others_beside_the_last_tile_of_two_warpgroups(cuda_device, n_q, T, N, causal):
    """Both warpgroups of a block of tokens end in one tile of keys, which holds the first keys of the next request: nothing of
    what those are reaches either's rows.  Requests of one warpgroup's rows stand between, so that the warpgroups of a
    multiprocessor are apart when they come to the tile."""
    B = 24
    q_lens, kv_lens = [T, 100] * B, [N, 120] * B
    c = Prefill(cuda_device, n_q, q_lens, kv_lens, seed=T, behind=140)
    mine = np.concatenate([np.arange(c.start[2 * b], c.start[2 * b + 1]) for b in range(B)])
    want = [x[mine] for x in c.run(causal)]
    ok(c.pool)
    ref, rl, tol, lt = prefill_ref(c.q, c.k, c.v, c.r, c.start[:2], c.kv_start[:2], causal, SCALE, cuda_device)
    assert_within(want[0][:T], ref[:T], tol[:T], "out")
    assert_within(want[1][:T], rl[:T], lt[:T], "lse")
    for bad in (float("nan"), float("inf"), -float("inf")):
        for b in range(B):   # the requests between, and (behind the last of them) rows of nobody
            c.v[c.kv_start[2 * b + 1]:c.kv_start[2 * b + 2]] = bad
        c.v[c.kv_start[-1]:] = bad
        for _ in range(3):
            got = c.run(causal)
            assert torch.equal(got[0][mine], want[0]) and torch.equal(got[1][mine], want[1])


def test_prefill_rows_of_nobody_behind_the_last_tile_of_two_warpgroups(cuda_device):
    """Room to spare behind the only request's keys, never written: with and without a mask."""
    for T, N, causal in ((200, 250, True), (254, 383, True), (200, 300, False), (256, 1, False)):
        c = Prefill(cuda_device, 64, [T], [N], seed=N, behind=300)
        want = c.run(causal)
        for x in (c.k, c.v, c.r):
            x[N:] = float("nan")
        for _ in range(5):
            got = c.run(causal)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n_q,gap,behind", [(3, 8, 8), (5, 24, 16), (1, 8, 40), (2, 0, 8)])
def test_prefill_strides_that_are_no_multiples(cuda_device, n_q, gap, behind):
    """Heads `gap` values apart and `behind` more behind a token's last: a token's stride is no multiple of a head's."""
    dev = cuda_device
    c = Prefill(dev, n_q, [140, 9], [200, 77], seed=n_q)
    want = c.run()

    def spread(x):
        n, h, d = x.shape
        wide = torch.full((n, h * (d + gap) + behind), float("nan"), dtype=torch.bfloat16, device=dev)
        y = wide.as_strided((n, h, d), (wide.shape[1], d + gap, 1))
        y.copy_(to(dev, x))
        return y

    r = torch.full((c.r.shape[0], ROT + behind), float("nan"), dtype=torch.bfloat16, device=dev)
    r[:, :ROT] = to(dev, c.r)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    kvd.kvd_latent_prefill(c.pool.handle, to(dev, c.q), to(dev, c.start), spread(c.k), spread(c.v), r[:, :ROT], to(dev, c.kv_start), out,
                           lse_out=lse)
    ok(c.pool)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_prefill_bad_pairs(cuda_device):
    dev = cuda_device
    for start, kv, skipped in (([0, 30, 20, 60], [0, 30, 60, 90], [1]), ([0, 20, 40, 61], [0, 30, 60, 90], [2]),
                               ([0, 20, 40, 60], [0, 30, 20, 90], [1]), ([0, 20, 40, 60], [-1, 30, 60, 91], [0, 2])):
        c = Prefill(dev, 2, [20, 20, 20], [30, 30, 30], seed=9)
        c.start, c.kv_start = np.array(start, np.int32), np.array(kv, np.int32)
        out, lse = c.run()
        oob(c.pool)
        good = [b for b in range(3) if b not in skipped]
        for b in good:
            e = Prefill(dev, 2, [20, 20, 20], [30, 30, 30], seed=9)
            e.start, e.kv_start = c.start[b:b + 2], c.kv_start[b:b + 2]
            ref, rl, tol, lt = e.ref()
            # (a broken pair in the middle leaves its neighbours' rows overlapping: those are either's)
            mine = [r for r in range(start[b], start[b + 1]) if sum(start[g] <= r < start[g + 1] for g in good) == 1]
            assert_within(out[mine], ref[mine], tol[mine], "out")
            assert_within(lse[mine], rl[mine], lt[mine], "lse")


def test_prefill_pieces_merge_to_the_whole(cuda_device):
    """Pieces of a prefix, not causal, and the chunk itself, causal, joined by their log-sum-exps."""
    dev, H, T, N = cuda_device, 4, 70, 400
    c = Prefill(dev, H, [T], [N], seed=10)
    whole = c.ref()
    parts = []
    for lo, hi, causal in ((0, 200, False), (200, 330, False), (330, 400, True)):
        d = Prefill(dev, H, [T], [N], seed=10)
        d.kv_start = np.array([lo, hi], np.int32)
        parts.append(d.run(causal))
    # a unit of kvd_combine_splits is a (row, KV head): 8 heads each; here every row is one of T "requests"
    o = torch.stack([x[0] for x in parts], 1).contiguous()       # [T][3][H][128]
    l = torch.stack([x[1] for x in parts], 1).contiguous()
    first = torch.arange(T, dtype=torch.int32, device=dev) * 3
    count = torch.full((T,), 3, dtype=torch.int32, device=dev)
    out = torch.empty(T, H, 128, dtype=torch.float32, device=dev)
    lse = torch.empty(T, H, dtype=torch.float32, device=dev)
    kvd.kvd_combine_splits(o, l, first, count, T, H, 1, out, lse)
    assert_within(out, whole[0], 2 * whole[2], "out")
    assert_within(lse, whole[1], 2 * whole[3], "lse")


def test_prefill_same_bits_and_graph(cuda_device):
    dev = cuda_device
    c = Prefill(dev, 6, [200, 30], [260, 900], seed=11)
    a, b = c.run(dtype=torch.bfloat16), c.run(dtype=torch.bfloat16)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q, st, ks = to(dev, c.q), to(dev, c.start), to(dev, c.kv_start)
    k, v, r = to(dev, c.k.contiguous()), to(dev, c.v.contiguous()), to(dev, c.r.contiguous())
    out, lse = torch.zeros_like(a[0]), torch.zeros_like(a[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvd.kvd_latent_prefill(c.pool.handle, q, st, k, v, r, ks, out, lse_out=lse)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a[0]) and torch.equal(lse, a[1])


# ------------------------------------------------------------------------ together
@KINDS
def test_a_prompt_in_chunks_and_its_decode(cuda_device, kind):
    """Append, read back, expand and attend chunk by chunk; then decode in the absorbed form.  Both forms and the plain
    softmax over the cached rows agree."""
    dev, H, rng = cuda_device, 8, np.random.default_rng(20)
    chunks, steps = [100, 37, 1], 3
    total = sum(chunks) + steps
    bt, nb = tables([total], 2, 1)
    pool = poisoned(1, nb, kind, dev)
    w_k = to(dev, rand(rng, H, 128, LAT, factor=LAT ** -0.5)).double()       # the expanding projections
    w_v = to(dev, rand(rng, H, 128, LAT, factor=LAT ** -0.5)).double()
    rope = kvd.Rope(ROT, 10000.0, interleaved=True, device=dev)
    norm = to(dev, (1.0 + 0.1 * rand(rng, LAT).float()).bfloat16())
    table = to(dev, bt)
    at = 0
    for T in chunks + [1] * steps:
        N = at + T
        x = to(dev, rand(rng, T, KEY))
        q = to(dev, rand(rng, T, H, 192))
        pos = torch.arange(at, N, dtype=torch.int32, device=dev)
        slots = to(dev, slots_of(bt, 0, at, N))
        kvd.kvd_latent_append(pool.handle, 0, x[:, :LAT], x[:, LAT:], slots, positions=pos, rope=rope, norm_weight=norm,
                              q_rope=q[..., 128:])
        start, kv_start = torch.tensor([0, T], dtype=torch.int32, device=dev), torch.tensor([0, N], dtype=torch.int32, device=dev)
        # expanded
        rows = torch.empty(N, KEY, dtype=torch.bfloat16, device=dev)
        kvd.kvd_latent_gather(pool.handle, 0, table, kv_start, rows)
        k = torch.einsum("hdc,nc->nhd", w_k, rows[:, :LAT].double()).bfloat16()
        v = torch.einsum("hdc,nc->nhd", w_v, rows[:, :LAT].double()).bfloat16()
        o1 = torch.empty(T, H, 128, dtype=torch.float32, device=dev)
        kvd.kvd_latent_prefill(pool.handle, q, start, k, v, rows[:, LAT:], kv_start, o1)
        # absorbed
        qa = torch.cat([torch.einsum("hdc,thd->thc", w_k, q[..., :128].double()), q[..., 128:].double()], -1).bfloat16()
        ws = torch.empty(kvd.kvd_latent_workspace_bytes(pool.handle, H, 1), dtype=torch.uint8, device=dev)
        oc = torch.empty(T, H, LAT, dtype=torch.float32, device=dev)
        kvd.kvd_latent_attn(pool.handle, 0, qa, start, table, torch.tensor([N], dtype=torch.int32, device=dev), ws, oc)
        o2 = torch.einsum("hdc,thc->thd", w_v, oc.double())
        ok(pool)
        # the formula over what the cache holds
        c = read_pool(pool)[0][0][slots_of(bt, 0, 0, N)].to(dev)
        seen = torch.arange(N, device=dev)[None] <= torch.arange(at, N, device=dev)[:, None]
        key = torch.cat([torch.einsum("hdc,nc->nhd", w_k, c[:, :LAT]), c[:, None, LAT:].expand(-1, H, -1)], -1)
        logit = torch.einsum("thd,nhd->thn", q.double(), key) * SCALE
        p = torch.softmax(torch.where(seen[:, None], logit, -torch.inf), -1)
        ref = torch.einsum("thn,nhd->thd", p, torch.einsum("hdc,nc->nhd", w_v, c[:, :LAT]))
        # k, v and the absorbed queries are rounded to bf16 here: each logit is off by 2^-8 of its products' size at most,
        # weights twice that and 2^-8 of their own, v by 2^-8 (the read-back of 8 bits by 2^-8 once more)
        size = torch.einsum("thd,nhd->thn", q.double().abs(), key.abs()) * SCALE
        wide = torch.einsum("thc,nc->thn", torch.cat([torch.einsum("hdc,thd->thc", w_k, q[..., :128].double()), q[..., 128:].double()],
                                                     -1).abs(), c.abs()) * SCALE
        vv = torch.einsum("hdc,nc->nhd", w_v, c[:, :LAT]).abs()
        va = torch.einsum("hdc,nc->nhd", w_v.abs(), c[:, :LAT].abs())
        for got, big in ((o1, torch.maximum(size, wide)), (o2, wide)):
            shift = (p * (torch.where(seen[:, None], big, 0.0) * 2.0 ** -7 * 1.1)).amax(-1, keepdim=True) + \
                torch.einsum("thn,thn->th", p, torch.where(seen[:, None], big, 0.0) * 2.0 ** -7 * 1.1)[..., None]
            rel = torch.where(seen[:, None], big, 0.0) * 2.0 ** -7 * 1.1
            tol = torch.einsum("thn,nhd->thd", p * (2 * rel + 2.0 ** -7), vv) + shift * ref.abs() + \
                torch.einsum("thn,nhd->thd", p, va) * 2.0 ** -7
            assert_within(got, ref, tol, "out")
        at = N


@KINDS
def test_copied_blocks(cuda_device, kind):
    """kvd_tier_move copies records: a request forked to blocks of its own attends the same."""
    dev = cuda_device
    c = Attn(dev, kind, 6, [1], [50], seed=21, layers=2, spare=6)
    want = c.run()
    free = np.setdiff1d(np.arange(c.nb), c.bt)[:4].astype(np.int32)
    kvd.kvd_tier_move(c.pool.handle, to(dev, c.bt[0].copy()), to(dev, free))
    c.bt[0] = free
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok(c.pool)


@pytest.mark.parametrize("op", ["append", "gather", "attn", "prefill"])
def test_another_current_device_is_refused(cuda_device, op):
    from test_latent_host import append_args, attn_args, call, gather_args, latent, prefill_args
    import ctypes

    torch.cuda.current_stream()
    pool = latent(device=torch.cuda.current_device() + 1)
    args = dict(append=append_args, gather=gather_args, attn=attn_args, prefill=prefill_args)[op]
    assert call("kvd_latent_" + op, args(pool=ctypes.byref(pool))) == kvd.KVD_ERR_INVALID


def test_rounding_constants():
    assert EPS[torch.bfloat16] == torch.finfo(torch.bfloat16).eps / 2 and EPS[torch.float32] == torch.finfo(torch.float32).eps / 2
