"""The latent cache's operators in 64 bits, from their formulas and the documented layout, with error bounds."""

import numpy as np
import torch

import paged_gqa_decode_kvd_gb300 as kvd

LAT, ROT, KEY = 512, 64, 576
EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # a rounding, relative: half a step


def places(fp8):
    """Element index of (token, dim) in a record: [16][576] bf16 values, or [16][512] bytes and [16][64] bf16 values."""
    t, d = np.arange(16)[:, None], np.arange(KEY)[None, :]
    if not fp8:
        return ((t // 8) * 9216 + (d // 64) * 1024 + (t % 8) * 128 + (((d % 64) // 8) ^ (t % 8)) * 16 + (d % 8) * 2) // 2
    c, e = d[:, :LAT], d[:, :ROT]
    return ((t // 8) * 4096 + (c // 64) * 512 + (t % 8) * 64 + c % 64,
            (8192 + (t // 8) * 1024 + (t % 8) * 128 + ((e // 8) ^ (t % 8)) * 16 + (e % 8) * 2) // 2)


def read_pool(pool):
    """(values [layers][blocks·16][576], codes' values, scales) in fp64 on the CPU; the last two None for bf16."""
    fp8 = pool.kv_dtype == kvd.KVD_LATENT_FP8
    rec = pool.mem.cpu().view(pool.num_layers, pool.num_blocks, pool.record_bytes)
    if not fp8:
        v = rec.view(torch.bfloat16).double()[..., torch.from_numpy(places(False))]
        return v.flatten(1, 2), None, None
    c, r = (torch.from_numpy(x) for x in places(True))
    code = rec[..., :8192].contiguous().view(torch.float8_e4m3fn).double()[..., c]
    rot = rec.view(torch.bfloat16).double()[..., r]
    scale = rec[..., 10240:].contiguous().view(torch.float32).double()
    return (torch.cat([code * scale[..., None], rot], -1).flatten(1, 2), code.flatten(1, 2), scale.flatten(1, 2))


def tables(lens, spare=3, seed=0):
    """int32 [B][most] shuffled distinct blocks (−1 behind a request's last), and the pool's blocks."""
    counts = [-(-max(n, 0) // 16) for n in lens]
    nb = sum(counts) + spare
    perm = np.random.default_rng(seed).permutation(nb).astype(np.int32)
    bt = np.full((len(lens), max(max(counts), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(counts):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, nb


def slots_of(bt, b, lo, hi):
    pos = np.arange(lo, hi)
    return (bt[b, pos // 16].astype(np.int64) * 16 + pos % 16)


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def softmax_rows(q, k, v, seen, scale, magnitude=None):
    """out, lse and their bounds for rows q [m][D] over keys k [n][D], values v [n][dv], seen [m][n]; fp64.

    The kernels' logit is an fp32 sum of D exact products (off by at most D + 8 steps of 2^-23 of the sum of their
    absolute values, whatever the order and whether steps are rounded or cut), scaled (one step more).  A weight: the logit's
    error twice (its own and its reference's), 2^-21 of the exponential, then 2^-8 once it is rounded to bf16; sums and
    products add 2^-23 a term."""
    logit = torch.where(seen, (q @ k.T) * scale, -torch.inf)
    size = abs(scale) * (q.abs() @ k.abs().T)
    delta = torch.where(seen, size, 0.0).amax(1) * (k.shape[1] + 8) * 2.0 ** -23 if k.shape[0] else torch.zeros(q.shape[0])
    lse = torch.logsumexp(logit, 1) if k.shape[0] else torch.full((q.shape[0],), -torch.inf, dtype=torch.float64)
    w = torch.exp(logit - torch.where(lse == -torch.inf, 0.0, lse)[:, None])
    vv = torch.where(v.isfinite(), v, 0.0)
    out = w @ vv
    for j in torch.nonzero(~v.isfinite().all(1)).flatten().tolist():   # reaches the rows that attend it, and no other
        odd = torch.where(v[j].isfinite(), 0.0, v[j])
        out = torch.where(seen[:, j, None], out + w[:, j, None] * odd, out)
    n = k.shape[0]
    rel = 2.0 ** -8 + 4.0 * delta + 2.0 ** -20 + n * 2.0 ** -23
    tol = (w @ vv.abs()) * rel[:, None]
    top = torch.where(seen, logit.abs(), 0.0).amax(1) if n else torch.zeros(q.shape[0])
    ltol = 2.0 * delta + 2.0 ** -20 + n * 2.0 ** -23 + (top + lse.abs().nan_to_num(posinf=0.0)) * 2.0 ** -21
    return out, lse, tol, ltol


def attn_ref(rows, q, start, bt, lens, retain, scale, device="cpu", absent=()):
    """Absorbed attention: rows [blocks·16][576] fp64, q [n][H][576]; absent: block ids that are not attended."""
    rows, q = rows.to(device), q.double().to(device)
    n, H, _ = q.shape
    out = torch.zeros(n, H, LAT, dtype=torch.float64, device=device)
    lse = torch.full((n, H), -torch.inf, dtype=torch.float64, device=device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, N in enumerate(lens):
        s0, T = int(start[b]), int(start[b + 1] - start[b])
        if T <= 0 or N < T:
            continue
        pos = np.arange(N)
        ids = bt[b, pos // 16].astype(np.int64)
        kept = ~np.isin(ids, absent)
        if retain is not None:
            kept &= (retain[np.where(kept, ids, 0)] >> (pos % 16) & 1).astype(bool)
        k = rows[torch.from_numpy(np.where(kept, ids * 16 + pos % 16, 0)).to(device)]
        k = torch.where(torch.from_numpy(kept).to(device)[:, None], k, 0.0)
        at = torch.arange(N, device=device)[None, :]
        limit = (N - T + torch.arange(T, device=device)).repeat_interleave(H)[:, None]
        seen = (at <= limit) & torch.from_numpy(kept).to(device)[None, :]
        o, l, t, lt = softmax_rows(q[s0:s0 + T].flatten(0, 1), k, k[:, :LAT], seen, scale)
        out[s0:s0 + T], lse[s0:s0 + T] = o.view(T, H, LAT), l.view(T, H)
        tol[s0:s0 + T], ltol[s0:s0 + T] = t.view(T, H, LAT), lt.view(T, H)
    return out, lse, tol, ltol


def prefill_ref(q, k, v, r, start, kv_start, causal, scale, device="cpu"):
    """Expanded attention: q [n][H][192], k, v [m][H][128], r [m][64]."""
    q, k, v, r = (x.double().to(device) for x in (q, k, v, r))
    n, H, _ = q.shape
    out = torch.zeros(n, H, 128, dtype=torch.float64, device=device)
    lse = torch.full((n, H), -torch.inf, dtype=torch.float64, device=device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(start) - 1):
        s0, T, k0, N = int(start[b]), int(start[b + 1] - start[b]), int(kv_start[b]), int(kv_start[b + 1] - kv_start[b])
        if T <= 0 or N <= 0:
            continue
        seen = torch.ones(T, N, dtype=torch.bool, device=device)
        if causal:
            seen = torch.arange(N, device=device)[None, :] <= N - T + torch.arange(T, device=device)[:, None]
        for h in range(H):
            key = torch.cat([k[k0:k0 + N, h], r[k0:k0 + N]], 1)
            (out[s0:s0 + T, h], lse[s0:s0 + T, h], tol[s0:s0 + T, h], ltol[s0:s0 + T, h]) = softmax_rows(
                q[s0:s0 + T, h], key, v[k0:k0 + N, h], seen, scale)
    return out, lse, tol, ltol


def assert_within(got, ref, tol, what, dtype=torch.float32):
    """|got − ref| ≤ tol and the rounding of got's type; infinities and NaN at the same places."""
    got, ref = got.double().cpu(), ref.cpu()
    tol = tol.cpu() + (ref.abs() + tol.cpu()).nan_to_num(posinf=0.0, neginf=0.0) * EPS[dtype] + 1e-38
    same = (got == ref) | (got.isnan() & ref.isnan())
    bad = ~same & ~((got - ref).abs() <= tol)
    if bool(bad.any()):
        i = int(torch.where(bad, ((got - ref).abs() / tol).nan_to_num(nan=torch.inf), 0.0).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst {got.flatten()[i]} for "
                             f"{ref.flatten()[i]} ± {tol.flatten()[i]} at {np.unravel_index(i, got.shape)}")
