"""Cases of the operators of a paged latent cache, with their plain forms.

A token's keys and values of all heads come from one latent vector of 512 values and 64 rotated ones.

  append   norm the latent, rotate the 64 dims of the key and of the queries, write the cache (bf16 or 8 bits)
  gather   read rows of the cache back as bf16, to expand them to the heads' keys and values
  attn     absorbed form: queries of 576 against the cached rows, values are their first 512
  prefill  expanded form: causal attention over every head's own 128 + 64 dims of key and 128 of value

A pool is one byte tensor in the layout that include/kvd.h documents, a record a block of 16 tokens.
Both forms read and write those bytes.
"""

import math
import random

import torch

own = False

DEV = "cuda"
BS = 16          # tokens per block
LAT = 512        # values of a latent vector
ROT = 64         # rotated dims, shared by the heads
NOPE = 128       # a head's own key dims in the expanded form
VD = 128         # a head's value dims in the expanded form
REC = {"bf16": 18432, "fp8": 10304}
SCALE = (NOPE + ROT) ** -0.5
EPS = 1e-6
# Base of the rotary frequencies.
BASE = 500000.0
# Elements of a block of logits: 8 GiB of them.
LOGITS = 1 << 31


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 32 requests: one token each, the smallest call
        dict(name="append-step", op="append", kind="bf16", tokens=32, n_q=32, norm=True, start=8191, mix=1),
        # a prompt's chunk in the middle of a long context into an 8-bit cache, an odd count of tokens
        dict(name="append-prompt-fp8", op="append", kind="fp8", tokens=4099, n_q=128, norm=True, start=61001, mix=2),
        # one request's cached prefix, to expand it for the next chunk of its prompt
        dict(name="gather-prefix", op="gather", kind="bf16", batch=1, len_lo=8192, len_hi=8192, skip=0, mix=3),
        # pieces of many requests' prefixes from an 8-bit cache, starting anywhere in a block
        dict(name="gather-ragged-fp8", op="gather", kind="fp8", batch=24, len_lo=100, len_hi=16384, skip=1000, mix=4),
        # one request's decode step, a short context: latency counts
        dict(name="attn-one", op="attn", kind="bf16", n_q=16, batch=1, q_lo=1, q_hi=1, ctx_lo=1019, ctx_hi=1019,
             evict=0.0, mix=5),
        # a batch's decode step, few heads (one part of a model split over several GPUs): the cache is streamed
        dict(name="attn-batch", op="attn", kind="bf16", n_q=16, batch=32, q_lo=1, q_hi=1, ctx_lo=8191, ctx_hi=8191,
             evict=0.0, mix=6),
        # the same with all of a large model's heads: as much arithmetic as memory traffic
        dict(name="attn-batch-wide", op="attn", kind="bf16", n_q=128, batch=32, q_lo=1, q_hi=1, ctx_lo=8191,
             ctx_hi=8191, evict=0.0, mix=7),
        # a serving step: single tokens next to drafted ones, ragged contexts, evicted slots
        dict(name="attn-ragged", op="attn", kind="bf16", n_q=32, batch=64, q_lo=1, q_hi=4, ctx_lo=256, ctx_hi=32768,
             evict=0.03, mix=8),
        # one request of 128k tokens in an 8-bit cache
        dict(name="attn-128k-fp8", op="attn", kind="fp8", n_q=64, batch=1, q_lo=1, q_hi=1, ctx_lo=131071,
             ctx_hi=131071, evict=0.0, mix=9),
        # a short prompt
        dict(name="prefill-short", op="prefill", n_q=8, batch=1, q_lo=77, q_hi=77, ctx_lo=0, ctx_hi=0, mix=10),
        # a whole prompt in one chunk: the largest
        dict(name="prefill-whole", op="prefill", n_q=32, batch=1, q_lo=8192, q_hi=8192, ctx_lo=0, ctx_hi=0, mix=11),
        # prompts' chunks of many lengths, each behind the part of its prompt that is cached
        dict(name="prefill-ragged", op="prefill", n_q=40, batch=12, q_lo=33, q_hi=2048, ctx_lo=1, ctx_hi=8192, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "gather", "attn", "attn", "prefill"))
    mix = rng.randrange(1 << 30)
    kind = rng.choice(("bf16", "fp8"))
    if op == "append":
        return dict(op="append", kind=kind, tokens=_log(rng, 1, 7700), n_q=rng.choice((1, 4, 8, 20, 32, 64, 128)),
                    norm=rng.random() < 0.7, start=rng.randrange(0, 131072), mix=mix)
    if op == "gather":
        lo = _log(rng, 1, 4096)
        return dict(op="gather", kind=kind, batch=_log(rng, 1, 32), len_lo=lo, len_hi=lo + _log(rng, 1, 8192),
                    skip=rng.choice((0, 7, 1000)), mix=mix)
    while True:
        if op == "attn":
            c = dict(op="attn", kind=kind, n_q=rng.choice((1, 4, 8, 16, 20, 32, 64, 96, 128)), batch=_log(rng, 1, 64),
                     q_lo=1, q_hi=_log(rng, 1, 64), ctx_lo=_log(rng, 1, 512), ctx_hi=_log(rng, 512, 65536),
                     evict=rng.choice((0.0, 0.0, 0.03, 0.5)), mix=mix)
        else:
            c = dict(op="prefill", n_q=rng.choice((1, 4, 8, 20, 32, 64, 128)), batch=_log(rng, 1, 24), q_lo=1,
                     q_hi=_log(rng, 1, 4096), ctx_lo=1, ctx_hi=_log(rng, 1, 16384), mix=mix)
        if work(c)["flops"] < 6.0e11 and sum(_lengths(c)[1]) < 300000:
            return c


def _lengths(c):
    """(new tokens, context with them) of every request of an attention case."""
    r = random.Random(c["mix"])
    q = [_log(r, c["q_lo"], c["q_hi"]) for _ in range(c["batch"])]
    ctx = [_log(r, c["ctx_lo"], c["ctx_hi"]) if c["ctx_lo"] else c["ctx_hi"] for _ in range(c["batch"])]
    return q, [a + b for a, b in zip(q, ctx)]


def _gather_lens(c):
    """(first position, rows) of every request of a gather case."""
    r = random.Random(c["mix"])
    return [r.randint(0, c["skip"]) for _ in range(c["batch"])], [r.randint(c["len_lo"], c["len_hi"])
                                                                 for _ in range(c["batch"])]


def work(c):
    token = {"bf16": 1152.0, "fp8": 644.0}.get(c.get("kind"))
    if c["op"] == "append":
        n = c["tokens"]
        return {"bytes": n * (2.0 * (LAT + ROT) + token + c["n_q"] * 4.0 * ROT + 12),
                "flops": n * (4.0 * LAT + 3.0 * ROT * (c["n_q"] + 1))}
    if c["op"] == "gather":
        return {"bytes": sum(_gather_lens(c)[1]) * (token + 1152.0), "flops": 0}
    q, lens = _lengths(c)
    pairs = sum(t * (n - t) + t * (t + 1) // 2 for t, n in zip(q, lens)) * (1.0 - c.get("evict", 0.0))
    if c["op"] == "attn":
        return {"bytes": sum(lens) * (1.0 - c["evict"]) * token + sum(q) * c["n_q"] * (2.0 * (2 * LAT + ROT) + 4),
                "flops": 2.0 * (2 * LAT + ROT) * c["n_q"] * pairs}
    return {"bytes": sum(lens) * 2.0 * (c["n_q"] * (NOPE + VD) + ROT) + sum(q) * c["n_q"] * (2.0 * (NOPE + ROT + VD) + 4),
            "flops": 2.0 * (NOPE + ROT + VD) * c["n_q"] * pairs}


# ------------------------------------------------------------ pool layout
def _swizzle(rows):
    """[..., 16 tokens, 64·c dims] to the order of a record's bf16 pieces: [8-token half][c][8 tokens][8 pieces of 8],
    piece p of token t in place p ^ (t % 8).  Its own inverse on the last axes, see _unswizzle."""
    x = rows.unflatten(-2, (2, 8)).unflatten(-1, (-1, 8, 8))              # [2][8 t][c][8 p][8]
    x = x.movedim(-3, -4)                                                 # [2][c][8 t][8 p][8]
    return torch.gather(x, -2, _PIECE.to(x.device)[:, :, None].expand(x.shape)).flatten(-5)


def _unswizzle(flat):
    """The inverse: [..., 16·64·c] values to [..., 16 tokens, 64·c dims]."""
    x = flat.unflatten(-1, (2, -1, 8, 8, 8))
    x = torch.gather(x, -2, _PIECE.to(x.device)[:, :, None].expand(x.shape))
    return x.movedim(-4, -3).flatten(-3).flatten(-3, -2)


_PIECE = torch.arange(8)[:, None] ^ torch.arange(8)[None, :]


def _values(records, kind):
    """fp32 [..., 16, 576] of records [..., bytes]."""
    if kind == "bf16":
        return _unswizzle(records.view(torch.bfloat16)).float()
    codes, rot, scale = _parts(records)
    lat = codes.float().unflatten(-1, (2, 8, 8, 64)).movedim(-2, -3).flatten(-2).flatten(-3, -2)
    return torch.cat([lat * scale[..., None], _unswizzle(rot).float()], -1)


def _parts(records):
    """Views of 8-bit records: codes [..., 8192] (order [half][64 dims][8 tokens][64]), rotated dims, scales."""
    return (records[..., :8192].view(torch.float8_e4m3fn), records[..., 8192:10240].view(torch.bfloat16),
            records[..., 10240:].view(torch.float32))


def _records(rows, kind):
    """Bytes [..., record] of rows [..., 16, 576]."""
    if kind == "bf16":
        return _swizzle(rows.bfloat16()).view(torch.uint8)
    lat = rows[..., :LAT].float()
    scale = lat.abs().amax(-1) / 448.0
    codes = (lat / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = codes.unflatten(-2, (2, 8)).unflatten(-1, (8, 64)).movedim(-2, -3).flatten(-4)
    return torch.cat([codes, _swizzle(rows[..., LAT:].bfloat16()).view(torch.uint8), scale.view(torch.uint8)], -1)


# ------------------------------------------------------------------ inputs
def _generator(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    return g


def _table(counts, total, g):
    """int32 [batch][most]: counts[b] distinct blocks a request, shuffled over the pool."""
    perm = torch.randperm(total, generator=g, device=DEV).int()
    table = torch.full((len(counts), max(counts)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def _starts(counts):
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    return torch.tensor(starts, dtype=torch.int32, device=DEV)


def _pool_memory(blocks, kind, g):
    """Records of normed latents: dims of different sizes, as a trained norm's weights make them."""
    rows = torch.randn(blocks, BS, LAT + ROT, generator=g, device=DEV)
    rows *= torch.linspace(0.5, 1.5, LAT + ROT, device=DEV)
    return _records(rows, kind).reshape(-1)


class _Pool:
    """A pool handle that goes with the state."""

    def __init__(self, kvd, blocks, kind, mem):
        dtype = {"bf16": kvd.KVD_LATENT_BF16, "fp8": kvd.KVD_LATENT_FP8}[kind]
        self.kvd, self.handle = kvd, kvd.kvd_pool_create(1, 1, blocks, dtype, mem, d_h=LAT + ROT)

    def __del__(self):
        self.kvd.kvd_pool_destroy(self.handle)


def prepare(case, seed):
    g = _generator(case, seed)
    s = {"case": case}
    {"append": _prepare_append, "gather": _prepare_gather, "attn": _prepare_attn,
     "prefill": _prepare_prefill}[case["op"]](case, g, s)
    if own:
        import paged_gqa_decode_kvd_gb300 as kvd

        s["kvd"] = kvd
        s["pool"] = _Pool(kvd, s["blocks"], case.get("kind", "bf16"), s["mem"])
        if case["op"] == "append":
            s["rope"] = kvd.Rope(ROT, BASE, interleaved=True, device=DEV)
        elif case["op"] == "attn":
            n = kvd.kvd_latent_workspace_bytes(s["pool"].handle, case["n_q"], case["batch"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


def _prepare_append(c, g, s):
    n = c["tokens"]
    # one projection gives a token's latent and the rotated part of its key, another one all heads' queries
    x = torch.randn(n, LAT + ROT, generator=g, device=DEV).mul_(3.0).bfloat16()
    s["latent"], s["k_rope"] = x[:, :LAT], x[:, LAT:]
    s["q_rope"] = torch.randn(n, c["n_q"], NOPE + ROT, generator=g, device=DEV).bfloat16()[..., NOPE:]
    s["q_out"] = torch.zeros(n, c["n_q"], LAT + ROT, dtype=torch.bfloat16, device=DEV)[..., LAT:]
    s["norm"] = (1.0 + 0.2 * torch.randn(LAT, generator=g, device=DEV)).bfloat16() if c["norm"] else None
    if n <= 64:   # a decode step: every token its own request, blocks and positions all over the pool
        pos = torch.randint(0, c["start"] + 1, (n,), generator=g, device=DEV)
        block = torch.arange(n, device=DEV)
        s["blocks"] = n + 3
    else:
        pos = torch.arange(c["start"], c["start"] + n, device=DEV)
        block = pos // BS - c["start"] // BS
        s["blocks"] = (c["start"] + n - 1) // BS - c["start"] // BS + 4
    s["slots"] = torch.randperm(s["blocks"], generator=g, device=DEV)[block] * BS + pos % BS
    s["pos"] = pos.int()
    s["mem"] = _pool_memory(s["blocks"], c["kind"], g)


def _prepare_gather(c, g, s):
    first, rows = _gather_lens(c)
    counts = [-(-(a + n) // BS) for a, n in zip(first, rows)]
    s["blocks"] = sum(counts) + 3
    s["mem"] = _pool_memory(s["blocks"], c["kind"], g)
    s["table"] = _table(counts, s["blocks"], g)
    s["first"] = torch.tensor(first, dtype=torch.int32, device=DEV)
    s["starts"] = _starts(rows)
    s["out"] = torch.zeros(sum(rows), LAT + ROT, dtype=torch.bfloat16, device=DEV)


def _prepare_attn(c, g, s):
    q, lens = _lengths(c)
    counts = [-(-n // BS) for n in lens]
    s["blocks"] = sum(counts) + 3
    s["mem"] = _pool_memory(s["blocks"], c["kind"], g)
    s["table"] = _table(counts, s["blocks"], g)
    s["mask"] = None
    if c["evict"]:
        keep = torch.rand(s["blocks"], BS, generator=g, device=DEV) >= c["evict"]
        bits = (keep.int() << torch.arange(BS, device=DEV, dtype=torch.int32)).sum(1)
        s["mask"] = (bits - ((bits >> 15) << 16)).to(torch.int16)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["host"] = (q, lens)
    s["starts"] = _starts(q)
    s["q"] = torch.randn(sum(q), c["n_q"], LAT + ROT, generator=g, device=DEV).bfloat16()
    s["out"] = torch.zeros(sum(q), c["n_q"], LAT, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros(sum(q), c["n_q"], dtype=torch.float32, device=DEV)


def _prepare_prefill(c, g, s):
    q, lens = _lengths(c)
    s["host"] = (q, lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["starts"], s["kv_starts"] = _starts(q), _starts(lens)
    s["q"] = torch.randn(sum(q), c["n_q"], NOPE + ROT, generator=g, device=DEV).bfloat16()
    # one projection expands a latent to every head's key and value; the rotated dims stay in the gathered rows
    kv = torch.randn(sum(lens), c["n_q"], NOPE + VD, generator=g, device=DEV).bfloat16()
    s["k_nope"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
    s["k_rope"] = torch.randn(sum(lens), LAT + ROT, generator=g, device=DEV).bfloat16()[:, LAT:]
    s["out"] = torch.zeros(sum(q), c["n_q"], VD, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros(sum(q), c["n_q"], dtype=torch.float32, device=DEV)
    s["blocks"] = 1
    s["mem"] = torch.zeros(REC["bf16"], dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------- the pass
def run(s):
    return {"append": _run_append, "gather": _run_gather, "attn": _run_attn, "prefill": _run_prefill}[s["case"]["op"]](s)


def _pool_views(s):
    """A pool's contents as the values they stand for: bf16 values, or codes, rotated dims and scales."""
    kind = s["case"]["kind"]
    if kind == "bf16":
        return s["mem"].view(torch.bfloat16)
    return _parts(s["mem"].view(-1, REC["fp8"]))


def _rotate(x, cos, sin):
    """Neighbouring pairs of x [n][...][64] turned, in fp32."""
    a, b = x.float().unflatten(-1, (-1, 2)).unbind(-1)
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _run_append(s):
    if own:
        s["kvd"].kvd_latent_append(s["pool"].handle, 0, s["latent"], s["k_rope"], s["slots"], positions=s["pos"],
                                   rope=s["rope"], norm_weight=s["norm"], norm_eps=EPS, q_rope=s["q_rope"],
                                   q_rope_out=s["q_out"])
        return s["q_out"], _pool_views(s)
    kind = s["case"]["kind"]
    freq = BASE ** (-torch.arange(0, ROT, 2, dtype=torch.float64, device=DEV) / ROT)
    angle = s["pos"].double()[:, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    s["q_out"].copy_(_rotate(s["q_rope"], cos[:, None], sin[:, None]))
    rot = _rotate(s["k_rope"], cos, sin).bfloat16()
    lat = s["latent"].float()
    if s["norm"] is not None:
        lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * s["norm"].float()
    block, t = s["slots"] // BS, s["slots"] % BS
    piece = _PIECE.to(DEV)[t % 8]                                        # [n][8]
    if kind == "bf16":
        x = torch.cat([lat.bfloat16(), rot], -1).unflatten(-1, (9, 8, 8))
        mem = s["mem"].view(torch.bfloat16).view(-1, 2, 9, 8, 8, 8)
        mem[block, t // 8, :, t % 8] = torch.gather(x, 2, piece[:, None, :, None].expand(x.shape))
        return s["q_out"], _pool_views(s)
    records = s["mem"].view(-1, REC["fp8"])
    scale = lat.abs().amax(-1) / 448.0
    scale = torch.where(scale == 0, 1.0, scale)
    codes = (lat / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).unflatten(-1, (8, 64))
    records[:, :8192].unflatten(1, (2, 8, 8, 64))[block, t // 8, :, t % 8] = codes
    x = rot.unflatten(-1, (8, 8))
    place = records[:, 8192:10240].view(torch.bfloat16).unflatten(1, (2, 8, 8, 8))
    place[block, t // 8, t % 8] = torch.gather(x, 1, piece[:, :, None].expand(x.shape))
    records[:, 10240:].view(torch.float32)[block, t] = scale
    return s["q_out"], _pool_views(s)


def _run_gather(s):
    if own:
        s["kvd"].kvd_latent_gather(s["pool"].handle, 0, s["table"], s["starts"], s["out"], first=s["first"])
        return s["out"]
    kind = s["case"]["kind"]
    row = torch.arange(s["out"].shape[0], device=DEV)
    b = torch.searchsorted(s["starts"], row, right=True) - 1
    pos = (row - s["starts"][b] + s["first"][b]).long()
    slot = s["table"].long()[b, pos // BS] * BS + pos % BS
    rows = _values(s["mem"].view(-1, REC[kind]), kind).reshape(-1, LAT + ROT)
    return rows[slot].bfloat16()


def _attend(s, rows, heads, keys_of):
    """out, lse: softmax attention of every request's rows over its keys, in fp32; neighbouring requests side by side,
    padded, where that is not much more work and the logits leave room.  keys_of(b0, b1, most): K, V [b][h or 1][most][dims], kept."""
    q, lens = s["host"]
    rows_all = s["out"].shape[0]
    out = s["out"].new_zeros(rows_all + 1, *s["out"].shape[1:])                 # the last row takes the padding's
    lse = s["lse"].new_zeros(rows_all + 1, heads)
    q_lens = s["starts"][1:] - s["starts"][:-1]
    b0 = 0
    while b0 < len(q):
        b1 = b0 + 1
        while b1 < len(q):
            padded = (b1 + 1 - b0) * max(q[b0:b1 + 1]) * max(lens[b0:b1 + 1])
            real = sum(t * n for t, n in zip(q[b0:b1 + 1], lens[b0:b1 + 1]))
            if heads * padded > LOGITS or padded > max(2 * real, 1 << 16):
                break
            b1 += 1
        most_q, most = max(q[b0:b1]), max(lens[b0:b1])
        k, v, kept = keys_of(b0, b1, most)
        t, n = q_lens[b0:b1, None], s["lens"][b0:b1, None]
        at = torch.arange(most, device=DEV)
        step = max(1, LOGITS // ((b1 - b0) * heads * most))
        for i in range(0, most_q, step):
            i_q = torch.arange(i, min(i + step, most_q), device=DEV)[None, :]
            real = i_q < t
            idx = torch.where(real, s["starts"][b0:b1, None] + i_q, rows_all).long()
            x = rows[idx.clamp(max=rows_all - 1)].float().transpose(1, 2)                               # [b][h][rows][dims]
            m = x.shape[2]
            seen = kept[:, None, :] & (at <= (n - t + i_q)[..., None]) & (at < n)[:, None, :]
            if k.shape[1] == 1:                                                 # one key for all heads: one product
                logit = (x.flatten(1, 2) @ k[:, 0].mT).unflatten(1, (heads, m))
            else:
                logit = x @ k.mT
            logit = (logit * SCALE).masked_fill_(~seen[:, None], -math.inf)
            top = logit.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, 0.0, top)
            p = logit.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            if v.shape[1] == 1:
                o = (p.flatten(1, 2) @ v[:, 0]).unflatten(1, (heads, m))
            else:
                o = p @ v
            o = o / torch.where(total == 0, 1.0, total)
            out[idx] = o.transpose(1, 2).to(out.dtype)
            lse[idx] = (top + total.log())[..., 0].transpose(1, 2)
            del logit, p, seen, o
        b0 = b1
    return out[:-1], lse[:-1]


def _run_attn(s):
    c = s["case"]
    if own:
        s["kvd"].kvd_latent_attn(s["pool"].handle, 0, s["q"], s["starts"], s["table"], s["lens"], s["workspace"],
                                 s["out"], retain_mask=s["mask"], softmax_scale=SCALE, lse_out=s["lse"])
        return s["out"], s["lse"]
    records = s["mem"].view(-1, REC[c["kind"]])
    slot = torch.arange(BS, device=DEV)

    def keys_of(b0, b1, most):
        ids = s["table"][b0:b1, :-(-most // BS)].long().clamp(min=0)
        k = _values(records[ids], c["kind"]).flatten(1, 2)[:, :most]
        if s["mask"] is None:
            kept = torch.ones(k.shape[:2], dtype=torch.bool, device=DEV)
        else:
            kept = ((s["mask"][ids].int()[..., None] >> slot) & 1).bool().flatten(1)[:, :most]
        return k[:, None], k[:, None, :, :LAT], kept

    return _attend(s, s["q"], c["n_q"], keys_of)


def _run_prefill(s):
    c = s["case"]
    if own:
        s["kvd"].kvd_latent_prefill(s["pool"].handle, s["q"], s["starts"], s["k_nope"], s["v"], s["k_rope"],
                                    s["kv_starts"], s["out"], softmax_scale=SCALE, lse_out=s["lse"])
        return s["out"], s["lse"]

    def keys_of(b0, b1, most):
        at = s["kv_starts"][b0:b1, None] + torch.arange(most, device=DEV)
        at = at.clamp(max=s["v"].shape[0] - 1).long()
        rope = s["k_rope"][at][:, :, None].expand(-1, -1, c["n_q"], -1)
        k = torch.cat([s["k_nope"][at], rope], -1).float().transpose(1, 2)
        return k, s["v"][at].float().transpose(1, 2), torch.ones(at.shape, dtype=torch.bool, device=DEV)

    return _attend(s, s["q"], c["n_q"], keys_of)


# ------------------------------------------- the operators in 64 bits
def _places(kind):
    """[16][576] (or [16][512], [16][64]) element index of (token, dim) in a record, from the layout's formulas."""
    t, d = torch.arange(BS, device=DEV)[:, None], torch.arange(LAT + ROT, device=DEV)[None, :]
    if kind == "bf16":
        byte = (t // 8) * 9216 + (d // 64) * 1024 + (t % 8) * 128 + (((d % 64) // 8) ^ (t % 8)) * 16 + (d % 8) * 2
        return byte // 2
    lat, rot = d[:, :LAT], d[:, :ROT]
    return ((t // 8) * 4096 + (lat // 64) * 512 + (t % 8) * 64 + lat % 64,
            ((t // 8) * 1024 + (t % 8) * 128 + ((rot // 8) ^ (t % 8)) * 16 + (rot % 8) * 2) // 2)


def _exact_rows(s, slots):
    """fp64 [n][576] of slots block·16 + offset."""
    kind = s["case"]["kind"]
    block, t = slots.div(BS, rounding_mode="floor"), slots.remainder(BS)
    if kind == "bf16":
        return s["mem"].view(torch.bfloat16)[(block * (REC["bf16"] // 2))[:, None] + _places("bf16")[t]].double()
    codes, rot = _places("fp8")
    base = block * REC["fp8"]
    code = s["mem"][base[:, None] + codes[t]].view(torch.float8_e4m3fn).double()
    scale = s["mem"].view(torch.float32)[(base + 10240) // 4 + t].double()
    return torch.cat([code * scale[:, None],
                      s["mem"].view(torch.bfloat16)[((base + 8192) // 2)[:, None] + rot[t]].double()], 1)


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return {"append": _exact_append, "gather": _exact_gather, "attn": _exact_attn,
            "prefill": _exact_prefill}[case["op"]](case, s)


def _exact_append(c, s):
    turn = s["pos"].double()[:, None] * torch.exp(-math.log(BASE) / ROT * torch.arange(0, ROT, 2, device=DEV).double())
    turn = torch.polar(torch.ones_like(turn), turn)

    def rotated(x, by):
        z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous()) * by
        return torch.view_as_real(z).flatten(-2)

    q, rot = rotated(s["q_rope"], turn[:, None]), rotated(s["k_rope"], turn)
    lat = s["latent"].double()
    if s["norm"] is not None:
        lat = lat / torch.sqrt((lat * lat).sum(-1, keepdim=True) / LAT + EPS) * s["norm"].double()
    block, t = s["slots"].div(BS, rounding_mode="floor"), s["slots"].remainder(BS)
    if c["kind"] == "bf16":
        mem = s["mem"].view(torch.bfloat16).double()
        mem[(block * (REC["bf16"] // 2))[:, None] + _places("bf16")[t]] = torch.cat([lat, rot], 1)
        return q, mem
    codes, rots, scales = (x.double() for x in _parts(s["mem"].view(-1, REC["fp8"])))
    code_at, rot_at = _places("fp8")
    scale = lat.abs().max(-1).values / 448.0
    codes[block[:, None], code_at[t]] = lat / scale[:, None]
    rots[block[:, None], rot_at[t]] = rot
    scales[block, t] = scale
    return q, (codes, rots, scales)


def _exact_gather(c, s):
    starts, first = s["starts"].tolist(), s["first"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for b, a in enumerate(first):
        pos = torch.arange(a, a + starts[b + 1] - starts[b], device=DEV)
        out[starts[b]:starts[b + 1]] = _exact_rows(s, s["table"][b].long()[pos >> 4] * BS + (pos & 15))
    return out


def _exact_softmax(s, b, h, k, v, kept, out, lse):
    """Head h's (or heads h's) rows of request b over keys [n][dims], values [n][dims], 64 bits."""
    starts = s["starts"].tolist()
    t, n = starts[b + 1] - starts[b], k.shape[0]
    for i in range(0, t, 1024):
        r = slice(starts[b] + i, starts[b] + min(i + 1024, t))
        logit = torch.einsum("m...d,nd->m...n", s["q"][r, h].double(), k) / math.sqrt(NOPE + ROT)
        late = torch.arange(n, device=DEV)[None, :] - torch.arange(i, min(i + 1024, t), device=DEV)[:, None] > n - t
        hide = late | ~kept[None, :]
        logit = torch.where(hide[:, None] if logit.dim() == 3 else hide, -math.inf, logit)
        z = torch.logsumexp(logit, -1)
        p = torch.exp(logit - torch.where(z == -math.inf, 0.0, z)[..., None])
        out[r, h] = torch.einsum("m...n,nd->m...d", p, v)
        lse[r, h] = z


def _exact_attn(c, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        pos = torch.arange(n, device=DEV)
        ids = s["table"][b].long()[pos >> 4]
        rows = _exact_rows(s, ids * BS + (pos & 15))
        kept = torch.ones(n, dtype=torch.bool, device=DEV)
        if s["mask"] is not None:
            kept = s["mask"].long().remainder(1 << 16)[ids].div(2 ** (pos & 15), rounding_mode="floor").remainder(2) > 0
        _exact_softmax(s, b, slice(None), rows, rows[:, :LAT], kept, out, lse)
    return out, lse


def _exact_prefill(c, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    at = s["kv_starts"].tolist()
    for b in range(c["batch"]):
        r = slice(at[b], at[b + 1])
        kept = torch.ones(at[b + 1] - at[b], dtype=torch.bool, device=DEV)
        for h in range(c["n_q"]):
            k = torch.cat([s["k_nope"][r, h], s["k_rope"][r]], 1).double()
            _exact_softmax(s, b, h, k, s["v"][r, h].double(), kept, out, lse)
    return out, lse
