"""Latent attention with fp32 outputs: weights to 2^-15 of themselves (a bf16, cut off or rounded, and what it left of them,
rounded), not to the 2^-8 of one bf16.

Queries, keys and codes are small numbers whose products sum up exactly in fp32, so that what a logit is off by is its few
roundings (the scale's, products', the sum's: below 8 of them, 2^-24 each) and the weights' own rounding shows."""

import numpy as np
import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from latent_ref import KEY, LAT, ROT, assert_within, read_pool, slots_of, softmax_rows, starts, tables

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("kind", [kvd.KVD_LATENT_BF16, kvd.KVD_LATENT_FP8], ids=["bf16", "fp8"])


def fine(q, k, v, seen, scale):
    """softmax_rows with the bounds of a weight that is two bf16."""
    out, lse, _, ltol = softmax_rows(q, k, v, seen, scale)
    size = softmax_rows(q, k, v.abs(), seen, scale)[0]
    top = torch.where(seen, (q @ k.T).abs() * abs(scale), 0.0).amax(1, keepdim=True)
    # the weight's rounding; its logit's and its reference's; an exponential and a quotient; n sums
    return out, lse, size * (2.0 ** -15 + 2 * top * 2.0 ** -21 + 2.0 ** -20 + k.shape[0] * 2.0 ** -23), ltol


def pick(rng, *shape, of=(-2.0, -1.0, 0.0, 1.0, 2.0)):
    return torch.from_numpy(rng.choice(np.array(of), shape)).bfloat16()


@pytest.mark.parametrize("n_q,q_lens,kv_lens", [(3, [1, 40], [17, 40]), (2, [200], [250]), (5, [129, 1], [140, 64]), (16, [2] * 20, [33] * 20)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** -5, -2.0 ** -6])
def test_prefill(cuda_device, n_q, q_lens, kv_lens, causal, scale):
    dev, rng = cuda_device, np.random.default_rng(n_q)
    start, kv_start = starts(q_lens), starts(kv_lens)
    n, m = int(start[-1]), int(kv_start[-1])
    q, k, r = pick(rng, n, n_q, 192), pick(rng, m, n_q, 128), pick(rng, m, ROT)
    v = torch.from_numpy(rng.standard_normal((m, n_q, 128))).bfloat16()
    pool = kvd.LatentPool(1, 1, device=dev)
    out, lse = torch.zeros(n, n_q, 128, device=dev), torch.zeros(n, n_q, device=dev)
    kvd.kvd_latent_prefill(pool.handle, q.to(dev), torch.from_numpy(start).to(dev), k.to(dev), v.to(dev), r.to(dev),
                           torch.from_numpy(kv_start).to(dev), out, causal=causal, softmax_scale=scale, lse_out=lse)
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
    for b, (T, N) in enumerate(zip(q_lens, kv_lens)):
        rows, keys = slice(start[b], start[b + 1]), slice(kv_start[b], kv_start[b + 1])
        seen = torch.ones(T, N, dtype=torch.bool)
        if causal:
            seen = torch.arange(N)[None, :] <= N - T + torch.arange(T)[:, None]
        for h in range(n_q):
            key = torch.cat([k[keys, h], r[keys]], 1).double()
            ref, rl, tol, lt = fine(q[rows, h].double(), key, v[keys, h].double(), seen, scale)
            assert_within(out[rows, h], ref, tol, "out")
            assert_within(lse[rows, h], rl, lt, "lse")


@KINDS
@pytest.mark.parametrize("n_q,q_lens,lens", [(16, [1], [9]), (128, [1, 2], [40, 64]), (5, [2, 20], [300, 33]), (64, [1] * 3, [2000, 77, 900]),
                                             (20, [4], [1500]), (3, [1] * 40, list(range(1, 81, 2)))])
@pytest.mark.parametrize("scale", [2.0 ** -4, -2.0 ** -5])
def test_attn(cuda_device, kind, n_q, q_lens, lens, scale):
    dev, rng = cuda_device, np.random.default_rng(n_q + len(lens))
    bt, nb = tables(lens, 2, n_q)
    pool = kvd.LatentPool(1, nb, kind, device=dev)
    pool.mem.fill_(0xFF)
    for b, n in enumerate(lens):
        # fourteenths of a token's largest value, whose codes, multiples of 32 up to 448, 8 bits hold exactly
        lat = pick(rng, n, LAT, of=(0.0, 0.5, 1.0, -1.0, 1.5, -2.0, 3.0, -4.0)).double()
        lat[:, 5] = 7.0
        lat = (lat * torch.from_numpy(rng.choice([0.25, 0.3, 0.35, 0.5], (n, 1)) if kind == kvd.KVD_LATENT_FP8 else np.full((n, 1), 0.25))).bfloat16()
        kvd.kvd_latent_append(pool.handle, 0, lat.to(dev), pick(rng, n, ROT).to(dev), torch.from_numpy(slots_of(bt, b, 0, n)).to(dev))
    start = starts(q_lens)
    m = int(start[-1])
    q = pick(rng, m, n_q, KEY, of=(-1.0, 0.0, 0.0, 1.0))
    out, lse = torch.zeros(m, n_q, LAT, device=dev), torch.zeros(m, n_q, device=dev)
    ws = torch.empty(kvd.kvd_latent_workspace_bytes(pool.handle, n_q, len(lens)), dtype=torch.uint8, device=dev)
    kvd.kvd_latent_attn(pool.handle, 0, q.to(dev), torch.from_numpy(start).to(dev), torch.from_numpy(bt).to(dev),
                        torch.tensor(lens, dtype=torch.int32, device=dev), ws, out, softmax_scale=scale, lse_out=lse)
    assert kvd.kvd_get_device_error(pool.handle) == kvd.KVD_OK
    rows, codes, _ = read_pool(pool)
    if kind == kvd.KVD_LATENT_FP8:
        assert bool((codes[0][slots_of(bt, 0, 0, lens[0])] % 32 == 0).all())
    for b, (T, N) in enumerate(zip(q_lens, lens)):
        k = rows[0][slots_of(bt, b, 0, N)]
        mine = slice(start[b], start[b + 1])
        seen = (torch.arange(N)[None, :] <= N - T + torch.arange(T)[:, None]).repeat_interleave(n_q, 0)
        ref, rl, tol, lt = fine(q[mine].double().flatten(0, 1), k, k[:, :LAT], seen, scale)
        assert_within(out[mine].flatten(0, 1), ref, tol, "out")
        assert_within(lse[mine].flatten(), rl, lt, "lse")
