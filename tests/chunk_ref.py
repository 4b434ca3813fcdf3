"""Plain 64-bit forms of the chunk operators and the small pools their tests use."""

from __future__ import annotations

import math

import numpy as np
import torch

import oracle
import paged_gqa_decode_kvd_gb300 as kvd

KINDS = {"bf16": (kvd.KVD_BF16, 0), "fp8": (kvd.KVD_FP8_E4M3, 0), "mixed": (kvd.KVD_MIXED, 0),
         "angle": (kvd.KVD_ANGLE, 0), "int4": (kvd.KVD_INT4, 32), "int4g128": (kvd.KVD_INT4, 128),
         "int2": (kvd.KVD_INT2, 64), "int2g32": (kvd.KVD_INT2, 32)}
FORMATS = (kvd.KVD_BF16, kvd.KVD_FP8_E4M3, kvd.KVD_FP8_E5M2)
BF16_HALF = 2.0 ** -8    # bf16: half a step, relative


def make_pool(kind, layers, n_kv, blocks, dev, fill=0xFF, seed=0):
    """A device pool (every byte `fill`: 0xFF makes unwritten slots NaN) and, mixed, its block formats."""
    dtype, group = KINDS[kind]
    pool = kvd.KVPool(layers, n_kv, blocks, dtype, device=dev, group_size=group)
    pool.mem.fill_(fill)
    fmt = None
    if kind == "mixed":
        fmt = np.random.default_rng(seed).integers(0, 3, blocks).astype(np.uint8)
        pool.set_block_formats(torch.tensor([FORMATS[f] for f in fmt], dtype=torch.uint8, device=dev))
    return pool, fmt


def make_oracle(kind, n_kv, blocks, fmt=None):
    dtype, group = KINDS[kind]
    if kind == "mixed":
        return oracle.OraclePool(blocks, n_kv, 128, 16, block_fmt=fmt)
    if group:
        return oracle.OraclePool(blocks, n_kv, 128, 16, lowbit=(4 if dtype == kvd.KVD_INT4 else 2, group))
    return oracle.OraclePool(blocks, n_kv, 128, 16, fp8=kind == "fp8", angle=kind == "angle")


def tables(lens, spare, seed, width=0):
    """(int32 table [B][most] of distinct shuffled blocks, number of blocks)."""
    counts = [-(-n // 16) for n in lens]
    nb = sum(counts) + spare
    perm = np.random.default_rng(seed).permutation(nb)
    bt = np.full((len(lens), max(counts + [1, width])), -1, np.int32)
    at = 0
    for b, n in enumerate(counts):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, nb


def slots_of(bt, b, a, z):
    pos = np.arange(a, z)
    return bt[b, pos // 16].astype(np.int64) * 16 + pos % 16


def chunk_ref(k, v, q, q_start, bt, lens, retain, scale, lowbit=False):
    """(out, lse, bound on |out error|, bound on |lse error|) in fp64.

    k, v: fp64 [blocks][n_kv][16][128] as attention reads them; q fp64 [n][n_q][128].  Bounds, per value:
    the fp32 sum of 128 products is off by at most 128·2^-24 of the sum of their magnitudes, for each of the
    two or three roundings a product and its place in the sum see: δ = 2^-16·max_t scale·Σ|q||k| (plus 2^-8 of
    it where the key itself is rounded to bf16); each weight is then off by 2δ, by the bf16 rounding of the
    weight (2^-8) and 2^-20 for exp2 and the sums; the output by its own rounding."""
    n, n_q, _ = q.shape
    n_kv = k.shape[1]
    g = n_q // n_kv
    out, lse = np.zeros_like(q), np.full((n, n_q), -np.inf)
    tol, ltol = np.zeros_like(q), np.zeros((n, n_q))
    for b in range(len(lens)):
        s0, s1 = int(q_start[b]), int(q_start[b + 1])
        for h in range(n_kv):
            nb = -(-lens[b] // 16)
            ids = bt[b, :nb]
            kk = k[ids, h].reshape(-1, 128)
            vv = v[ids, h].reshape(-1, 128)
            keep = np.ones(nb * 16, bool)
            if retain is not None:
                keep = ((retain[ids].astype(np.int64)[:, None] >> np.arange(16)) & 1).astype(bool).reshape(-1)
            for i in range(s0, s1):
                sel = keep & (np.arange(nb * 16) <= lens[b] - (s1 - s0) + i - s0)
                if not sel.any():
                    continue
                for hq in range(h * g, h * g + g):
                    x = kk[sel] @ q[i, hq] * scale
                    m = x.max()
                    w = np.exp(x - m)
                    tot = w.sum()
                    lse[i, hq] = m + math.log(tot)
                    w /= tot
                    out[i, hq] = w @ vv[sel]
                    size = abs(scale) * (np.abs(kk[sel]) @ np.abs(q[i, hq])).max()
                    delta = size * (2.0 ** -16 + (BF16_HALF if lowbit else 0.0))
                    mass = w @ np.abs(vv[sel])
                    tol[i, hq] = mass * (2 * delta + BF16_HALF * (2 if lowbit else 1) + 2.0 ** -20) + \
                        BF16_HALF * np.abs(out[i, hq]) + 1e-30
                    ltol[i, hq] = delta + 2.0 ** -20 * (1 + abs(lse[i, hq]))
    return out, lse, tol, ltol


def assert_within(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities differ"
    err = np.abs(got[~inf] - ref[~inf])
    lim = tol[~inf]
    assert not np.isnan(err).any(), f"{what}: NaN"
    bad = err > lim
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside the bound, worst ratio {(err / lim).max():.3f}"


def rope_freqs_ref(rot, base, scaling="plain", factor=1.0, original_len=0.0, low=1.0, high=1.0):
    """(θ [rot/2] fp64, m), from the rules' formulas."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    th = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    m = 1.0
    if scaling == "linear":
        th = [t / factor for t in th]
    if scaling == "banded":
        out = []
        for t in th:
            w = min(max((original_len * t / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            out.append(w * t + (1 - w) * t / factor)
        th = out
    if scaling == "yarn":
        def pair(u):
            return rot * math.log(original_len / (2 * math.pi * u)) / (2 * math.log(base))
        a, z = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        out = []
        for j, t in enumerate(th):
            r = min(max((j - a) / max(z - a, 0.001), 0.0), 1.0)
            out.append((1 - r) * t + r * t / factor)
        th, m = out, 0.1 * math.log(factor) + 1
    return np.array(th), m


def rotate_ref(x, pos, theta, m, rot, interleaved):
    """fp64 rotation of x [n][h][128]; also the sum of magnitudes each output has (for bounds)."""
    y, size = x.copy(), np.zeros_like(x)
    ang = pos[:, None].astype(np.float64) * theta[None, :]
    c, s = np.cos(ang)[:, None, :] * m, np.sin(ang)[:, None, :] * m
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = (np.abs(a) + np.abs(b)) * abs(m)
    return y, size
