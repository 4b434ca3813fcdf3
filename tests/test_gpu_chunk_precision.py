"""Chunk attention keeps the output tolerance of the framework's attention whatever the number of rows in the call."""

import numpy as np
import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from chunk_ref import KINDS, tables
from harness import assert_out_close
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu


def reference(c, dev):
    """(out, lse, Σ w·|v|, max_t scale·Σ|q||k|) in fp64, by request and KV head."""
    k, v = (torch.from_numpy(x).to(dev) for x in c.opool.values())
    q = c.q.double()
    if c.kind == "angle":
        import oracle
        q = torch.from_numpy(oracle.angle_query(c.q.float().numpy())).double()
    q = q.to(dev)
    n, n_q, _ = q.shape
    g = n_q // c.n_kv
    out, mass, size = (torch.zeros_like(q) for _ in range(3))
    lse = torch.full((n, n_q), -np.inf, dtype=torch.float64, device=dev)
    for b, m in enumerate(c.lens):
        s0, s1 = int(c.start[b]), int(c.start[b + 1])
        if s1 == s0:
            continue
        ids = torch.from_numpy(c.bt[b, :-(-m // 16)].astype(np.int64)).to(dev)
        seen = torch.arange(m, device=dev)[None, :] <= torch.arange(m - (s1 - s0), m, device=dev)[:, None]
        if c.retain is not None:
            bits = c.retain[c.bt[b, :-(-m // 16)]].astype(np.int64)
            keep = ((bits[:, None] >> np.arange(16)) & 1).astype(bool).reshape(-1)[:m]
            seen = seen & torch.from_numpy(keep).to(dev)[None, :]
        for h in range(c.n_kv):
            kk, vv = k[ids, h].reshape(-1, 128)[:m], v[ids, h].reshape(-1, 128)[:m]
            x = q[s0:s1, h * g:h * g + g]
            l = torch.einsum("tgd,nd->tgn", x, kk) * 128 ** -0.5
            l = l.masked_fill(~seen[:, None, :], -np.inf)
            z = torch.logsumexp(l, -1)
            w = torch.exp(l - torch.where(torch.isneginf(z), 0.0, z)[..., None])
            out[s0:s1, h * g:h * g + g] = torch.einsum("tgn,nd->tgd", w, vv)
            mass[s0:s1, h * g:h * g + g] = torch.einsum("tgn,nd->tgd", w, vv.abs())
            lse[s0:s1, h * g:h * g + g] = z
            big = torch.einsum("tgd,nd->tgn", x.abs(), kk.abs()) * 128 ** -0.5
            size[s0:s1, h * g:h * g + g] = big.masked_fill(~seen[:, None, :], 0.0).amax(-1, keepdim=True)
    return out, lse, mass, size


def short_contexts(dev, kind, requests=160, seed=70):
    """Contexts of 1 to 48 positions, every position a row: few weights a row, so that their roundings do not average
    out, and far more than 1,024 rows."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, 49, requests)
    return Case(dev, kind, 16, 2, lens, lens, seed=seed)


@pytest.mark.parametrize("kind", sorted(k for k in KINDS if not k.startswith("int")))
def test_a_large_call_keeps_the_weights_precision(cuda_device, kind):
    """A weight is the sum of two bf16.  bf16 is off by at most 2^-8 relative, so the sum by at most 2^-16.  The weight's
    logit is off by δ = 2^-16·max_t scale·Σ|q||k| (fp32 sums of 128 products, as in chunk_ref), and so the weight by 2δ
    relative with the normalisation; exp2, the scale of an 8-bit record and the sums add 2^-19."""
    c = short_contexts(cuda_device, kind)
    assert c.q.shape[0] * c.n_q > 1024
    out, lse = c.run()
    ref, rlse, mass, size = reference(c, cuda_device)
    err = (out.double() - ref).abs()
    tol = mass * (2 * 2.0 ** -16 * size + 2.0 ** -16 + 2.0 ** -19)
    bad = err > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside the bound, worst ratio {(err / tol).max().item():.1f}"
    assert bool(((lse.double() - rlse).abs() <= 2.0 ** -16 * size[..., 0] + 2.0 ** -20 * (1 + rlse.abs())).all())
    assert_out_close(out.double().cpu().numpy(), ref.cpu().numpy())


@pytest.mark.parametrize("kind", sorted(k for k in KINDS if k.startswith("int")))
def test_low_bit_records_keep_their_precision(cuda_device, kind):
    """code·scale + zero, an fp32 value, enters the products as the sum of two bf16: off by 2^-16 of itself, which moves a
    logit by 2^-16·scale·Σ|q||k| more and an output by 2^-16·Σ w·|v| more than exact K and V do.  The product of a
    weight's second part (2^-7 of it) and a value's (2^-8) is left out: 2^-15·Σ w·|v|."""
    c = short_contexts(cuda_device, kind)
    out, lse = c.run()
    ref, rlse, mass, size = reference(c, cuda_device)
    err = (out.double() - ref).abs()
    tol = mass * (2 * 2.0 ** -15 * size + 2 * 2.0 ** -16 + 2.0 ** -15 + 2.0 ** -19)
    bad = err > tol
    outside = int((err > 2e-3 + 1e-2 * ref.abs()).sum())
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside the bound, worst ratio " \
        f"{(err / tol).max().item():.1f}; {outside} outside the output tolerance"
    assert bool(((lse.double() - rlse).abs() <= 2.0 ** -15 * size[..., 0] + 2.0 ** -20 * (1 + rlse.abs())).all())
    assert_out_close(out.double().cpu().numpy(), ref.cpu().numpy())


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_request_is_as_exact_in_a_batch_as_alone(cuda_device, kind):
    """The same bound for a request of few rows, in a call of its own and beside rows of no request."""
    c = Case(cuda_device, kind, 8, 2, [3], [30], seed=71)
    ref, _, mass, size = reference(c, cuda_device)
    tol = mass * (2 * 2.0 ** -16 * size + 2.0 ** -16 + 2.0 ** -19)
    d = c.device()
    alone = c.run(d=d)[0]
    d["q"] = torch.cat([d["q"], torch.zeros(200, 8, 128, dtype=torch.bfloat16, device=cuda_device)])
    beside = c.run(d=d)[0][:3]
    for got in (alone, beside):
        assert bool(((got.double() - ref).abs() <= tol).all())
    assert torch.equal(alone, beside)


def bad_value(c, pos, dim, value):
    """Position pos of request 0 is written again with one bad element in V; its K stays what it was."""
    blk, t = int(c.bt[0, pos // 16]), pos % 16
    k, v = (torch.from_numpy(x[blk, :, t].copy()).bfloat16()[None].to(c.dev) for x in c.opool.values())
    v[0, :, dim] = value
    kvd.kvd_append_kv(c.pool.handle, c.layer, k, v, torch.tensor([blk * 16 + t], device=c.dev))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("q_len,n_q", [(40, 4), (20, 1), (300, 4)])
@pytest.mark.parametrize("kind", ["bf16", "mixed"])
def test_a_cached_infinity_stays_one(cuda_device, kind, q_len, n_q, value):
    """An infinity in V ahead of the new tokens: every row attends it with a weight above zero, so the sum is that
    infinity (no weight times infinity is NaN unless the weight is 0), in its dim only."""
    c = Case(cuda_device, kind, n_q, 1, [q_len], [q_len + 260], seed=72)
    wide = range(260) if kind == "bf16" else \
        [p for p in range(260) if np.random.default_rng(72).integers(0, 3, c.nb)[c.bt[0, p // 16]] == 0]
    for pos in (wide[0], wide[len(wide) // 2], wide[-1]):
        bad_value(c, pos, 77, value)
        out, lse = c.run()
        ref, rlse, _, size = reference(c, cuda_device)
        hit = out[..., 77]
        assert bool(torch.isnan(hit).all() if np.isnan(value) else (hit == value).all())
        rest = [d for d in range(128) if d != 77]
        assert_out_close(out.double().cpu().numpy()[..., rest], ref.cpu().numpy()[..., rest])
        assert bool(((lse.double() - rlse).abs() <= 2.0 ** -16 * size[..., 0] + 2.0 ** -20 * (1 + rlse.abs())).all())
        bad_value(c, pos, 77, c.opool.values()[1][int(c.bt[0, pos // 16]), 0, pos % 16, 77])


@pytest.mark.parametrize("kind", ["bf16", "mixed"])
def test_infinities_that_cancel_are_nan(cuda_device, kind):
    c = Case(cuda_device, kind, 4, 1, [40], [300], seed=73)
    fmt = np.random.default_rng(73).integers(0, 3, c.nb)
    wide = [p for p in range(260) if kind == "bf16" or fmt[c.bt[0, p // 16]] == 0]
    bad_value(c, wide[0], 5, float("inf"))
    bad_value(c, wide[-1], 5, float("-inf"))
    out, _ = c.run()
    assert bool(torch.isnan(out[..., 5]).all()) and bool(torch.isfinite(out[..., 6:]).all())


@pytest.mark.parametrize("seed", [74, 75, 76])
@pytest.mark.parametrize("kind", ["bf16", "mixed"])
def test_bad_values_in_several_new_tiles_of_a_warpgroup(cuda_device, kind, seed):
    """128 rows behind 70 positions: four tiles, the last three with new tokens, two of them of the warpgroup that adds
    its bad values to its sums in tensor memory before the two are joined.  Each bad V reaches its own row and the later
    ones, in its own dim."""
    def formats(x):   # of the request's blocks in a mixed pool
        bt, nb = tables([198], 3, x)
        return np.random.default_rng(x).integers(0, 3, nb)[bt[0]]

    while kind == "mixed" and not (formats(seed)[12] == 0 and (formats(seed)[5:8] == 0).any()):
        seed += 100   # 16-bit blocks in the second and the fourth tile
    c = Case(cuda_device, kind, 1, 1, [128], [198], seed=seed)
    fmt = np.random.default_rng(seed).integers(0, 3, c.nb)
    wide = [p for p in range(70, 198) if kind == "bf16" or fmt[c.bt[0, p // 16]] == 0]
    clean, rlse, _, size = reference(c, cuda_device)
    values = [float("inf"), float("-inf"), float("nan")]
    pick = [next((p for p in wide if a <= p < z), None) for a, z in ((70, 100), (100, 128), (128, 160), (160, 192), (192, 198))]
    bad = {}
    for i, pos in enumerate(p for p in pick if p is not None):
        bad[pos] = (20 * i + 3, values[i % 3])
        bad_value(c, pos, *bad[pos])
    assert len(bad) >= (5 if kind == "bf16" else 2)
    out, lse = c.run()
    rest = [d for d in range(128) if d not in {x[0] for x in bad.values()}]
    assert_out_close(out.double().cpu().numpy()[..., rest], clean.cpu().numpy()[..., rest])
    for pos, (dim, value) in bad.items():
        row = pos - 70
        if row:
            assert_out_close(out[:row, 0, dim].double().cpu().numpy(), clean[:row, 0, dim].cpu().numpy())
        hit = out[row:, 0, dim]
        assert bool(torch.isnan(hit).all() if np.isnan(value) else (hit == value).all())
    assert bool(((lse.double() - rlse).abs() <= 2.0 ** -16 * size[..., 0] + 2.0 ** -20 * (1 + rlse.abs())).all())


def test_calls_back_to_back(cuda_device):
    """Calls of several kinds and sizes one behind the other, each block of one taking over an SM from the call before
    as soon as that leaves it: the same bits as alone."""
    cases = [Case(cuda_device, kind, n_q, n_kv, q, n, seed=77 + i) for i, (kind, n_q, n_kv, q, n) in enumerate([
        ("bf16", 4, 1, [3], [70]), ("fp8", 8, 1, [100], [300]), ("int4", 4, 2, [40, 1], [90, 500]), ("bf16", 16, 2, [65], [65]),
        ("mixed", 4, 1, [1], [5]), ("angle", 4, 1, [20], [400])])]
    data = [c.device() for c in cases]
    alone = []
    for c, d in zip(cases, data):
        alone.append(c.run(d=d))
        torch.cuda.synchronize()
    got = [[c.run(d=d) for c, d in zip(cases, data)] for _ in range(30)]
    torch.cuda.synchronize()
    for turn in got:
        for (a, x), (b, y) in zip(alone, turn):
            assert torch.equal(a, b) and torch.equal(x, y)
    for c in cases:
        assert kvd.kvd_get_device_error(c.pool.handle) == kvd.KVD_OK
