"""Cases of three operators of the paged KV cache, with their plain forms.

  chunk    causal attention of a chunk of new tokens of every request over its paged cache
  rope     rotary positions of a chunk's queries and keys, and the append of its K and V
  compact  the retained slots of a batch copied to dense blocks, the evicted ones left behind

A pool is one byte tensor in the layout that include/kvd.h documents, [layer][block][KV head]
records of a K tile, a V tile and (8-bit) 32 fp32 scales.  Both forms read and write those bytes.
"""

import math
import random

import torch

own = False

DEV = "cuda"
D = 128          # head dimension
BS = 16          # tokens per block
REC = {"bf16": 8192, "fp8": 4224}
# Base of the rotary frequencies.
BASE = 500000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # four drafted tokens of one request checked at once: the smallest call, latency counts
        dict(name="chunk-draft", op="chunk", kind="bf16", n_q=32, n_kv=8, batch=1, q_lo=4, q_hi=4, ctx_lo=1019,
             ctx_hi=1019, evict=0.0, mix=1),
        # the same for a batch with long contexts: the cache is streamed once
        dict(name="chunk-draft-batch", op="chunk", kind="bf16", n_q=32, n_kv=8, batch=32, q_lo=5, q_hi=5,
             ctx_lo=8187, ctx_hi=8187, evict=0.0, mix=2),
        # one chunk of a long prompt behind the part that is in the cache
        dict(name="chunk-prompt", op="chunk", kind="bf16", n_q=32, n_kv=8, batch=1, q_lo=2048, q_hi=2048,
             ctx_lo=8192, ctx_hi=8192, evict=0.0, mix=3),
        # a whole prompt in one chunk: nothing cached before it
        dict(name="chunk-whole-prompt", op="chunk", kind="bf16", n_q=32, n_kv=8, batch=1, q_lo=8192, q_hi=8192,
             ctx_lo=0, ctx_hi=0, evict=0.0, mix=4),
        # a serving step: prompts of every length next to single tokens, ragged, with evicted slots
        dict(name="chunk-serving", op="chunk", kind="bf16", n_q=28, n_kv=4, batch=48, q_lo=1, q_hi=900, ctx_lo=1,
             ctx_hi=16384, evict=0.03, mix=5),
        # the last chunk of a 128k context in an 8-bit cache, 8 query heads a KV head: the largest
        dict(name="chunk-128k-fp8", op="chunk", kind="fp8", n_q=64, n_kv=8, batch=1, q_lo=512, q_hi=512,
             ctx_lo=130560, ctx_hi=130560, evict=0.0, mix=6),
        # a decode step of 32 requests: one token each
        dict(name="rope-step", op="rope", tokens=32, n_q=32, n_kv=8, rot=128, interleaved=False, scaling="banded",
             start=8191, fused=True, mix=7),
        # a prompt of 8,192 tokens, q, k and v as slices of one projection
        dict(name="rope-prompt", op="rope", tokens=8192, n_q=32, n_kv=8, rot=128, interleaved=False,
             scaling="banded", start=0, fused=True, mix=8),
        # half of each head, neighbours paired, far positions, an odd count that starts inside a block
        dict(name="rope-partial", op="rope", tokens=4099, n_q=64, n_kv=8, rot=64, interleaved=True, scaling="yarn",
             start=126973, fused=False, mix=9),
        # two short requests and few layers
        dict(name="compact-short", op="compact", kind="bf16", layers=4, n_kv=8, batch=2, len_lo=777, len_hi=800,
             evict=0.1, mix=10),
        # a batch of reasoning traces in every layer, a few slots evicted here and there
        dict(name="compact-traces", op="compact", kind="bf16", layers=28, n_kv=4, batch=8, len_lo=7000, len_hi=8192,
             evict=0.03, mix=11),
        # one long request of a deep model in an 8-bit cache, a third evicted
        dict(name="compact-long-fp8", op="compact", kind="fp8", layers=80, n_kv=8, batch=1, len_lo=16411,
             len_hi=16411, evict=0.33, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "rope", "compact"))
    mix = rng.randrange(1 << 30)
    n_kv = rng.choice((1, 2, 4, 8))
    if op == "chunk":
        while True:
            c = dict(op="chunk", kind=rng.choice(("bf16", "bf16", "fp8")), n_q=n_kv * rng.choice((1, 2, 4, 5, 7, 8)),
                     n_kv=n_kv, batch=_log(rng, 1, 48), q_lo=1, q_hi=_log(rng, 1, 4096), ctx_lo=_log(rng, 1, 512),
                     ctx_hi=_log(rng, 512, 65536), evict=rng.choice((0.0, 0.0, 0.03, 0.5)), mix=mix)
            if work(c)["flops"] < 1.0e12 and sum(_lengths(c)[1]) < 600000:
                return c
    if op == "rope":
        return dict(op="rope", tokens=_log(rng, 1, 8192), n_q=n_kv * rng.choice((1, 2, 4, 5, 7, 8)), n_kv=n_kv,
                    rot=2 * rng.randint(8, 64), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(("plain", "linear", "ntk", "banded", "yarn")), start=rng.randrange(0, 131072),
                    fused=rng.random() < 0.5, mix=mix)
    while True:
        lo = _log(rng, 1, 8192)
        c = dict(op="compact", kind=rng.choice(("bf16", "fp8")), layers=_log(rng, 1, 80), n_kv=n_kv,
                 batch=_log(rng, 1, 32), len_lo=lo, len_hi=lo + _log(rng, 1, 8192),
                 evict=rng.choice((0.01, 0.1, 0.5, 0.9)), mix=mix)
        if work(c)["bytes"] < 6.0e9:
            return c


def _lengths(c):
    """(new tokens, context with them) of every request of a chunk case."""
    r = random.Random(c["mix"])
    q = [_log(r, c["q_lo"], c["q_hi"]) for _ in range(c["batch"])]
    ctx = [_log(r, c["ctx_lo"], c["ctx_hi"]) if c["ctx_lo"] else c["ctx_hi"] for _ in range(c["batch"])]
    return q, [a + b for a, b in zip(q, ctx)]


def _compact_lens(c):
    r = random.Random(c["mix"])
    return [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["batch"])]


def work(c):
    if c["op"] == "chunk":
        q, lens = _lengths(c)
        pairs = sum(t * (n - t) + t * (t + 1) // 2 for t, n in zip(q, lens)) * (1.0 - c["evict"])
        per = 512 if c["kind"] == "bf16" else 264
        return {"bytes": sum(lens) * (1.0 - c["evict"]) * c["n_kv"] * per + sum(q) * c["n_q"] * (2 * 2 * D + 4),
                "flops": 4.0 * D * c["n_q"] * pairs}
    if c["op"] == "rope":
        n = c["tokens"]
        return {"bytes": n * (c["n_q"] * 4.0 * D + c["n_kv"] * 8.0 * D + 12),
                "flops": 3.0 * n * (c["n_q"] + c["n_kv"]) * c["rot"]}
    per = 512 if c["kind"] == "bf16" else 264
    kept = sum(_compact_lens(c)) * (1.0 - c["evict"])
    return {"bytes": 2.0 * kept * c["layers"] * c["n_kv"] * per, "flops": 0}


# ------------------------------------------------------------ pool layout
# Axes of a tile's elements in memory: the 16 dims of a group i are c8·8 + x·2 + c1 (K) or r8·8 + r7 (V),
# the 16 tokens of a block t8·8 + t7 (K) or t8·8 + x·2 + t1 (V); an 8-bit tile pairs the groups i.
_AXES = {("bf16", 0): ((8, 8, 4, 2, 2, 2), (4, 1, 0, 3, 2, 5)), ("bf16", 1): ((8, 8, 4, 2, 2, 2), (3, 2, 5, 0, 4, 1)),
         ("fp8", 0): ((4, 8, 4, 2, 2, 2, 2), (5, 1, 0, 3, 4, 2, 6)),
         ("fp8", 1): ((4, 8, 4, 2, 2, 2, 2), (4, 2, 6, 0, 3, 5, 1))}


def _rows(tile, kind, side):
    """A tile's elements [..., 2048] as [..., 16 tokens, 128 dims] (side 0: K, 1: V)."""
    shape, order = _AXES[kind, side]
    lead = tile.dim() - 1
    t = tile.reshape(*tile.shape[:-1], *shape)
    t = t.permute(*range(lead), *[lead + a for a in order])
    return t.reshape(*tile.shape[:-1], BS, D)


def _tile(rows, kind, side):
    """The inverse: [..., 16, 128] to the tile's order [..., 2048]."""
    shape, order = _AXES[kind, side]
    lead = rows.dim() - 2
    back = [order.index(a) for a in range(len(order))]
    t = rows.reshape(*rows.shape[:-2], *[shape[a] for a in order])
    t = t.permute(*range(lead), *[lead + a for a in back])
    return t.reshape(*rows.shape[:-2], BS * D)


def _values(records, kind):
    """fp32 (K, V), each [..., 16, 128], of records [..., bytes]."""
    if kind == "bf16":
        e = records.view(torch.bfloat16).unflatten(-1, (2, BS * D))
        return tuple(_rows(e[..., s, :], kind, s).float() for s in (0, 1))
    e = records[..., :2 * BS * D].view(torch.float8_e4m3fn).unflatten(-1, (2, BS * D))
    scale = records[..., 2 * BS * D:].contiguous().view(torch.float32).unflatten(-1, (2, BS))
    return tuple(_rows(e[..., s, :].view(torch.uint8), kind, s).view(torch.float8_e4m3fn).float()
                 * scale[..., s, :, None] for s in (0, 1))


# ------------------------------------------------------------------ inputs
def _generator(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    return g


def _tables(counts, total, g, first=0):
    """int32 [batch][most]: counts[b] distinct blocks a request, shuffled over the ids from `first` on."""
    perm = (torch.randperm(total, generator=g, device=DEV) + first).int()
    table = torch.full((len(counts), max(counts)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def _mask(blocks, evict, g):
    """int16 [blocks] of retain bits, or None: every slot evicted with probability `evict`."""
    if not evict:
        return None
    keep = torch.rand(blocks, BS, generator=g, device=DEV) >= evict
    bits = (keep.int() << torch.arange(BS, device=DEV, dtype=torch.int32)).sum(1)
    return (bits - ((bits >> 15) << 16)).to(torch.int16)


def prepare(case, seed):
    g = _generator(case, seed)
    s = {"case": case}
    if case["op"] == "chunk":
        _prepare_chunk(case, g, s)
    elif case["op"] == "rope":
        _prepare_rope(case, g, s)
    else:
        _prepare_compact(case, g, s)
    if own:
        import paged_gqa_decode_kvd_gb300 as kvd

        kind = {"bf16": kvd.KVD_BF16, "fp8": kvd.KVD_FP8_E4M3}[case.get("kind", "bf16")]
        s["kvd"] = kvd
        s["pool"] = _Pool(kvd, kvd.kvd_pool_create(case.get("layers", 1), case["n_kv"], s["blocks"], kind, s["mem"]))
        if case["op"] == "chunk":
            n = kvd.kvd_chunk_workspace_bytes(s["pool"].handle, case["n_q"], case["batch"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        elif case["op"] == "rope":
            s["rope"] = kvd.Rope(case["rot"], BASE, interleaved=case["interleaved"], device=DEV, **s["scaling"])
        else:
            n = kvd.kvd_compact_workspace_bytes(s["pool"].handle, case["batch"], s["table"].shape[1])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


class _Pool:
    """A pool handle that goes with the state."""

    def __init__(self, kvd, handle):
        self.kvd, self.handle = kvd, handle

    def __del__(self):
        self.kvd.kvd_pool_destroy(self.handle)


def _prepare_chunk(c, g, s):
    q, lens = _lengths(c)
    counts = [-(-n // BS) for n in lens]
    nb = sum(counts) + 3
    s["blocks"] = nb
    rows = torch.randn(nb, c["n_kv"], 2, BS, D, generator=g, device=DEV)
    # keys differ in size from head to head, as trained ones do
    rows[:, :, 0] *= torch.linspace(0.5, 2.0, c["n_kv"], device=DEV)[None, :, None, None]
    if c["kind"] == "bf16":
        rows = rows.bfloat16()
        mem = torch.stack([_tile(rows[:, :, 0], "bf16", 0), _tile(rows[:, :, 1], "bf16", 1)], 2).view(torch.uint8)
    else:
        scale = rows.abs().amax(-1) / 448.0
        codes = (rows / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        tiles = [_tile(codes[:, :, i], "fp8", i) for i in (0, 1)] + [scale.flatten(2).view(torch.uint8)]
        mem = torch.cat(tiles, 2)
    s["mem"] = mem.reshape(-1)
    s["table"] = _tables(counts, nb, g)
    s["mask"] = _mask(nb, c["evict"], g)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["host"] = (q, lens)
    starts = [0]
    for t in q:
        starts.append(starts[-1] + t)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["q"] = torch.randn(starts[-1], c["n_q"], D, generator=g, device=DEV).bfloat16()
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(starts[-1], c["n_q"], dtype=torch.float32, device=DEV)


_SCALINGS = {"plain": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=8.0),
             "banded": dict(scaling="banded", factor=8.0, original_len=8192, low=1.0, high=4.0),
             "yarn": dict(scaling="yarn", factor=16.0, original_len=8192, low=1.0, high=32.0)}


def _prepare_rope(c, g, s):
    n, n_q, n_kv = c["tokens"], c["n_q"], c["n_kv"]
    s["scaling"] = _SCALINGS[c["scaling"]]
    if c["fused"]:
        x = torch.randn(n, n_q + 2 * n_kv, D, generator=g, device=DEV).bfloat16()
        s["q"], s["k"], s["v"] = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    else:
        s["q"], s["k"], s["v"] = (torch.randn(n, h, D, generator=g, device=DEV).bfloat16()
                                  for h in (n_q, n_kv, n_kv))
    if n <= 64:   # a decode step: every token its own request, blocks and positions all over the pool
        pos = torch.randint(0, c["start"] + 1, (n,), generator=g, device=DEV)
        block = torch.arange(n, device=DEV)
        nb = n + 3
    else:
        pos = torch.arange(c["start"], c["start"] + n, device=DEV)
        block = pos // BS - c["start"] // BS
        nb = (c["start"] + n - 1) // BS - c["start"] // BS + 4
    s["blocks"] = nb
    perm = torch.randperm(nb, generator=g, device=DEV)
    s["slots"] = perm[block] * BS + pos % BS
    s["pos"] = pos.int()
    s["mem"] = torch.randn(nb * n_kv * 2 * BS * D, generator=g, device=DEV).bfloat16().view(torch.uint8)
    s["q_out"] = torch.zeros(n, n_q, D, dtype=torch.bfloat16, device=DEV)


def _prepare_compact(c, g, s):
    lens = _compact_lens(c)
    counts = [-(-n // BS) for n in lens]
    total = sum(counts)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["source_blocks"], s["blocks"] = total, 2 * total
    s["table"] = _tables(counts, total, g)
    s["new_table"] = _tables(counts, total, g, first=total)
    mask = _mask(2 * total, c["evict"], g)
    s["mask"] = mask
    s["mem"] = torch.randint(0, 256, (c["layers"] * 2 * total * c["n_kv"] * REC[c["kind"]],), generator=g, device=DEV,
                             dtype=torch.uint8)
    stride = max(lens)
    s["scores"] = torch.rand(c["batch"], stride, generator=g, device=DEV)
    s["new_scores"] = torch.zeros_like(s["scores"])
    s["new_lens"] = torch.zeros_like(s["lens"])


# ---------------------------------------------------------------- the pass
def run(s):
    return {"chunk": _run_chunk, "rope": _run_rope, "compact": _run_compact}[s["case"]["op"]](s)


def _run_chunk(s):
    if own:
        s["kvd"].kvd_chunk_attn(s["pool"].handle, 0, s["q"], s["starts"], s["table"], s["lens"], s["workspace"],
                                s["out"], retain_mask=s["mask"], lse_out=s["lse"])
        return s["out"], s["lse"]
    c = s["case"]
    n_q, n_kv = c["n_q"], c["n_kv"]
    g = n_q // n_kv
    records = s["mem"].view(-1, n_kv, REC[c["kind"]])
    out, lse = torch.zeros_like(s["q"]), torch.zeros_like(s["lse"])
    at = 0
    for b, (t, n) in enumerate(zip(*s["host"])):
        ids = s["table"][b, :-(-n // BS)].long()
        k, v = (x.transpose(0, 1).reshape(n_kv, -1, D)[:, :n] for x in _values(records[ids], c["kind"]))
        kept = torch.ones(n, dtype=torch.bool, device=DEV)
        if s["mask"] is not None:
            kept = ((s["mask"][ids].int()[:, None] >> torch.arange(BS, device=DEV)) & 1).bool().reshape(-1)[:n]
        q = s["q"][at:at + t].float().view(t, n_kv, g, D).transpose(0, 1)
        step = max(1, (1 << 30) // (n_kv * g * n))   # rows at a time: 4 GiB of logits
        for i in range(0, t, step):
            rows = q[:, i:i + step].reshape(n_kv, -1, D)
            m = rows.shape[1] // g
            pos = torch.arange(n - t + i, n - t + i + m, device=DEV).repeat_interleave(g)
            seen = kept[None, :] & (torch.arange(n, device=DEV)[None, :] <= pos[:, None])
            logit = (rows @ k.transpose(1, 2)) * D ** -0.5
            logit = logit.masked_fill_(~seen, -math.inf)
            top = logit.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, 0.0, top)
            p = logit.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = (p @ v) / torch.where(total == 0, 1.0, total)
            out[at + i:at + i + m] = o.view(n_kv, m, g, D).transpose(0, 1).reshape(m, n_q, D).to(out.dtype)
            lse[at + i:at + i + m] = (top + total.log()).view(n_kv, m, g).transpose(0, 1).reshape(m, n_q)
            del logit, p, seen
        at += t
    return out, lse


def _frequencies(rot, scaling="plain", factor=1.0, original_len=0, low=1.0, high=1.0):
    """(radians a position of every pair, in fp64, and the factor on cos and sin)."""
    j = torch.arange(0, rot, 2, dtype=torch.float64, device=DEV)
    base = BASE * factor ** (rot / (rot - 2.0)) if scaling == "ntk" else BASE
    f = base ** (-j / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "banded":   # pairs that turn less than `low` times over the original length are stretched
        turns = original_len * f / (2.0 * math.pi)
        w = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        return f * w + f / factor * (1.0 - w), 1.0
    if scaling == "yarn":     # the ramp runs over the pair's index between the two turn counts
        def pair(turns):
            return rot * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(BASE))

        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        ramp = ((j / 2.0 - a) / max(b - a, 0.001)).clamp(0.0, 1.0)
        return f / factor * ramp + f * (1.0 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rotate(x, cos, sin, rot, interleaved):
    """x [n][h][128] turned by cos, sin [n][1][rot/2] over its first `rot` dims, in fp32."""
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1).bfloat16()


def _run_rope(s):
    c = s["case"]
    if own:
        s["kvd"].kvd_rope_append(s["pool"].handle, 0, s["q"], s["k"], s["v"], s["pos"], s["rope"], s["slots"],
                                 s["q_out"])
        return s["q_out"], s["mem"].view(torch.bfloat16)
    freq, m = _frequencies(c["rot"], **s["scaling"])
    angle = s["pos"].double()[:, None] * freq
    cos, sin = (m * angle.cos()).float()[:, None], (m * angle.sin()).float()[:, None]
    q = _rotate(s["q"], cos, sin, c["rot"], c["interleaved"])
    k = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"])
    order = torch.arange(BS * D, device=DEV).view(BS, D)
    mem = s["mem"].view(torch.bfloat16).view(-1, 2 * BS * D)   # a row a record
    slot = s["slots"]
    record = (slot // BS)[:, None] * c["n_kv"] + torch.arange(c["n_kv"], device=DEV)
    for side, x in ((0, k), (1, s["v"])):
        place = torch.empty(BS * D, dtype=torch.int64, device=DEV)
        place[_tile(order, "bf16", side)] = torch.arange(BS * D, device=DEV)
        place = place.view(BS, D)[slot % BS] + side * BS * D
        mem[record[:, :, None], place[:, None, :]] = x
    return q, s["mem"].view(torch.bfloat16)


def _run_compact(s):
    c = s["case"]
    L, n_kv, rec, n_src = c["layers"], c["n_kv"], REC[c["kind"]], s["source_blocks"]
    pool = s["mem"].view(L, s["blocks"], n_kv, rec)
    if own:
        s["kvd"].kvd_compact(s["pool"].handle, s["table"], s["lens"], s["new_table"], s["new_lens"], s["workspace"],
                             retain_mask=s["mask"], scores=s["scores"], new_scores=s["new_scores"])
        return pool[:, n_src:], s["new_lens"], s["new_scores"], s["mask"]
    B, most = s["table"].shape
    slot = torch.arange(most * BS, device=DEV)
    ids = s["table"].long().clamp(min=0).repeat_interleave(BS, 1)                        # [B][slots]
    kept = (slot < s["lens"][:, None]) & ((s["mask"][ids].int() >> (slot % BS)) & 1).bool()
    rank = kept.cumsum(1) - 1
    b, at = kept.nonzero(as_tuple=True)
    to = rank[b, at]
    source = ids[b, at] * BS + at % BS
    target = s["new_table"].long()[b, to // BS] * BS + to % BS - n_src * BS
    new_lens = kept.sum(1).int()
    new_scores = torch.zeros_like(s["scores"])
    new_scores[b, to] = s["scores"][b, at]
    used = (slot[::BS] < new_lens[:, None]).nonzero(as_tuple=True)
    written = s["new_table"].long()[used] - n_src
    elem, parts = (torch.int16, 2) if c["kind"] == "bf16" else (torch.uint8, 2)
    tiles = 2 * BS * D * (2 if c["kind"] == "bf16" else 1)
    for side in range(parts):
        lo = side * tiles // 2
        rows = _rows(pool[:, :n_src, :, lo:lo + tiles // 2].view(elem), c["kind"], side)   # [L][nb][n_kv][16][128]
        rows = rows.transpose(2, 3).reshape(L, n_src * BS, n_kv, D)
        dense = torch.zeros_like(rows)
        dense[:, target] = rows[:, source]
        dense = dense.view(L, n_src, BS, n_kv, D).transpose(2, 3)[:, written]
        pool[:, n_src + written, :, lo:lo + tiles // 2] = _tile(dense, c["kind"], side).view(torch.uint8)
    if c["kind"] == "fp8":
        rows = pool[:, :n_src, :, tiles:].contiguous().view(torch.int32).view(L, n_src, n_kv, 2, BS)
        rows = rows.permute(0, 1, 4, 2, 3).reshape(L, n_src * BS, n_kv, 2)
        dense = torch.zeros_like(rows)
        dense[:, target] = rows[:, source]
        dense = dense.view(L, n_src, BS, n_kv, 2).permute(0, 1, 3, 4, 2)[:, written]
        pool[:, n_src + written, :, tiles:] = dense.flatten(-2).contiguous().view(torch.uint8)
    mask = s["mask"].clone()
    mask[n_src + written] = -1   # every slot of a written block is kept
    return pool[:, n_src:], new_lens, new_scores, mask


# ------------------------------------------- the operators in 64 bits
def _place(kind, side):
    """[16][128] element index of (token, dim) in a tile, from the formulas of the layout."""
    t = torch.arange(BS, device=DEV)[:, None]
    d = torch.arange(D, device=DEV)[None, :]
    i, c = d // 16, d % 16
    if side == 0:
        lane, e = 4 * (t % 8) + (c % 8) // 2, c % 2 + 2 * (t // 8) + 4 * (c // 8)
    else:
        lane, e = 4 * (c % 8) + (t % 8) // 2, t % 2 + 2 * (c // 8) + 4 * (t // 8)
    if kind == "fp8":
        return ((i // 2) * 32 + lane) * 16 + (i % 2) * 8 + e
    return (i * 32 + lane) * 8 + e


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "chunk":
        return _exact_chunk(case, s)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    return None, None, _exact_scores(case, s), None


def _exact_chunk(c, s):
    n_q, n_kv = c["n_q"], c["n_kv"]
    g = n_q // n_kv
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    out = torch.zeros(starts[-1], n_q, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(starts[-1], n_q, dtype=torch.float64, device=DEV)
    records = s["mem"].view(s["blocks"], n_kv, REC[c["kind"]])
    for b, n in enumerate(lens):
        t = starts[b + 1] - starts[b]
        ids = s["table"][b, :(n + BS - 1) // BS].long()
        if s["mask"] is None:
            bias = torch.zeros(n, dtype=torch.float64, device=DEV)
        else:
            bits = s["mask"][ids].long().remainder(1 << 16)
            on = torch.stack([bits.bitwise_and(1 << o) for o in range(BS)], 1).flatten()[:n]
            bias = torch.where(on > 0, 0.0, -math.inf).double()
        for h in range(n_kv):
            r = records[ids, h]
            if c["kind"] == "bf16":
                e = r.view(torch.bfloat16).double()
                k, v = (e[:, o * BS * D + _place("bf16", o)].reshape(-1, D)[:n] for o in (0, 1))
            else:
                e = r[:, :2 * BS * D].contiguous().view(torch.float8_e4m3fn).double()
                w = r[:, 2 * BS * D:].contiguous().view(torch.float32).double()
                k, v = ((e[:, o * BS * D + _place("fp8", o)] * w[:, o * BS:(o + 1) * BS, None]).reshape(-1, D)[:n]
                        for o in (0, 1))
            for i in range(0, t, 512):
                m = min(512, t - i)
                x = s["q"][starts[b] + i:starts[b] + i + m, h * g:(h + 1) * g].double()
                logit = torch.einsum("mgd,nd->mgn", x, k) / math.sqrt(D) + bias
                late = torch.arange(n, device=DEV)[None, :] - torch.arange(m, device=DEV)[:, None] > n - t + i
                logit = torch.where(late[:, None, :], -math.inf, logit)
                z = torch.logsumexp(logit, -1)
                p = torch.exp(logit - torch.where(z == -math.inf, 0.0, z)[..., None])
                out[starts[b] + i:starts[b] + i + m, h * g:(h + 1) * g] = torch.einsum("mgn,nd->mgd", p, v)
                lse[starts[b] + i:starts[b] + i + m, h * g:(h + 1) * g] = z
    return out, lse


def _exact_rope(c, s):
    rot = c["rot"]
    freq, m = _frequencies(rot, **s["scaling"])
    turn = torch.polar(torch.full((c["tokens"], 1, rot // 2), m, dtype=torch.float64, device=DEV),
                       (s["pos"].double().view(-1, 1) * freq).view(c["tokens"], 1, rot // 2))

    def rotated(x):
        x = x.double()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        z = torch.complex(a, b) * turn
        y = x.clone()
        if c["interleaved"]:
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    mem = s["mem"].view(torch.bfloat16).double().view(s["blocks"], c["n_kv"], 2, BS * D)
    block, t = s["slots"].div(BS, rounding_mode="floor"), s["slots"].remainder(BS)
    for h in range(c["n_kv"]):
        for side, x in ((0, rotated(s["k"][:, h:h + 1])), (1, s["v"][:, h:h + 1].double())):
            mem[block[:, None], h, side, _place("bf16", side)[t]] = x[:, 0]
    return rotated(s["q"]), mem.reshape(-1)


def _exact_scores(c, s):
    new = torch.zeros_like(s["scores"], dtype=torch.float64)
    table, mask = s["table"].cpu(), s["mask"].cpu()
    for b, n in enumerate(s["lens"].tolist()):
        word = mask[table[b, :(n + BS - 1) // BS].long()].long().remainder(1 << 16)
        on = torch.stack([word.bitwise_and(1 << o) for o in range(BS)], 1).flatten()[:n] > 0
        kept = s["scores"][b, :n].double()[on.to(DEV)]
        new[b, :kept.numel()] = kept
    return new
