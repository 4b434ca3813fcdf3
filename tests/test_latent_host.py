"""Host side of the latent cache: sizes, and every refusal before a launch."""

import ctypes

import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from test_chunk_checks import Reached, Tensor
from test_chunk_host import FakePool, P, fake, rope_args

INV, UNS, MEM = kvd.KVD_ERR_INVALID, kvd.KVD_ERR_UNSUPPORTED, kvd.KVD_ERR_NOMEM
BF16, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
FORMATS = [kvd.KVD_LATENT_BF16, kvd.KVD_LATENT_FP8]


def latent(kind=kvd.KVD_LATENT_BF16, blocks=8, layers=2, device=0):
    f = FakePool()
    f.desc = kvd._lib.PoolDesc(layers, 1, 576, 16, blocks, kind, 0)
    f.num_sms, f.device, f.mem = 152, device, 1 << 50
    f.layer_bytes = blocks * (10304 if kind == kvd.KVD_LATENT_FP8 else 18432)
    return f


@pytest.mark.parametrize("layers,blocks", [(1, 1), (3, 17)])
def test_bytes(layers, blocks):
    assert kvd.kvd_pool_bytes(layers, 1, blocks, kvd.KVD_LATENT_BF16, d_h=576) == (layers * blocks * 16 * 1152,) * 2
    assert kvd.kvd_pool_bytes(layers, 1, blocks, kvd.KVD_LATENT_FP8, d_h=576) == (
        layers * blocks * 16 * 644, layers * blocks * 16 * 640)


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("n_kv,d_h,block", [(2, 576, 16), (1, 128, 16), (1, 512, 16), (1, 576, 32)])
def test_other_shapes_are_refused(kind, n_kv, d_h, block):
    with pytest.raises(kvd.KvdError) as e:
        kvd.kvd_pool_bytes(1, n_kv, 4, kind, d_h=d_h, block_size=block)
    assert e.value.status == UNS


def test_a_pool_of_k_and_v_has_128_dims():
    with pytest.raises(kvd.KvdError) as e:
        kvd.kvd_pool_bytes(1, 1, 4, kvd.KVD_BF16, d_h=576)
    assert e.value.status == UNS


@pytest.mark.parametrize("kind", FORMATS)
def test_the_other_entry_points_refuse_a_latent_pool(kind):
    pool, lib, n, b = latent(kind), kvd.load(), ctypes.c_size_t(), ctypes.c_int()
    ref = ctypes.byref(pool)
    assert lib.kvd_append_kv(ref, 0, P(16), P(16), P(8), 1, None) == UNS
    assert lib.kvd_decode_workspace_bytes(ref, 4, 1, 16, 1, ctypes.byref(b), ctypes.byref(n)) == UNS
    assert lib.kvd_decode_attn(ref, 0, P(16), 4, None, None, P(4), 4, P(4), 1, 16, 1, None, 0.1, P(256), 1 << 30, P(16), 0, None,
                               None, 0, None, 0, None) == UNS
    assert lib.kvd_decode_attn_noalloc(ref, 0, P(16), 4, None, None, P(4), 4, P(4), 1, 16, 1, None, 0.1, P(16), 0, None, None, 0,
                                       None, 0, None) == UNS
    assert lib.kvd_decode_plan(ref, 4, P(4), 4, P(4), 1, 16, 1, None, P(256), 1 << 30, None) == UNS
    assert lib.kvd_rope_append(*rope_args(pool)) == UNS
    assert lib.kvd_chunk_workspace_bytes(ref, 4, 1, ctypes.byref(n)) == UNS
    assert lib.kvd_chunk_attn(ref, 0, P(16), 4, P(4), 3, P(4), 4, P(4), 1, None, 0.1, P(256), 1 << 40, P(1 << 20), 0, None,
                              None) == UNS
    assert lib.kvd_compact_workspace_bytes(ref, 1, 4, ctypes.byref(n)) == UNS
    assert lib.kvd_compact(ref, P(4), 4, P(64), 2, None, P(4), 4, P(128), None, 8, None, 8, P(256), 1 << 20, None) == UNS
    assert lib.kvd_pool_attach_host_tier(ref, P(16), 1 << 30, None, 0, 4) == UNS
    assert lib.kvd_pool_set_block_formats(ref, P(16), 100) == INV
    with pytest.raises(kvd.KvdError):
        kvd.kvd_tier_bytes(1, 1, 8, kind, 4, d_h=576)


def call(name, a):
    return getattr(kvd.load(), name)(*a.values())


def append_args(**kw):
    a = dict(pool=ctypes.byref(latent()), layer=0, latent=P(1 << 20), ls=576, k=P((1 << 20) + 1024), ks=576, norm=P(1 << 16),
             eps=1e-6, q=P(1 << 22), qs=768, qh=192, n_q=4, pos=P(4), rope=kvd._lib.RopeDesc(4096, 64, 0, 1.0), slots=P(8), n=3,
             out=P(1 << 24), os=2304, oh=576, stream=None)
    a.update(kw)
    return a


def rope_desc(rot=64, inter=0, turns=4096):
    return kvd._lib.RopeDesc(turns, rot, inter, 1.0)


@pytest.mark.parametrize("bad,status", [
    (dict(pool=None), INV), (dict(pool=ctypes.byref(fake())), UNS), (dict(layer=2), INV), (dict(layer=-1), INV),
    (dict(n=-1), INV), (dict(n_q=-1), INV), (dict(n_q=257, qs=1 << 16, os=1 << 18), UNS), (dict(latent=None), INV),
    (dict(k=None), INV), (dict(slots=None), INV), (dict(pos=None), INV), (dict(q=None), INV), (dict(out=None), INV),
    (dict(rope=None), INV), (dict(rope=rope_desc(65)), INV), (dict(rope=rope_desc(0)), INV), (dict(rope=rope_desc(66)), UNS),
    (dict(rope=rope_desc(inter=2)), INV), (dict(rope=rope_desc(turns=None)), INV), (dict(rope=rope_desc(turns=4100)), INV),
    (dict(latent=P((1 << 20) + 8)), INV), (dict(k=P((1 << 20) + 1026)), INV), (dict(norm=P((1 << 16) + 2)), INV),
    (dict(ls=504), INV), (dict(ls=580), INV), (dict(ks=56), INV), (dict(ks=68), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(qs=636), INV), (dict(qs=632), INV), (dict(qh=56), INV), (dict(qh=196), INV),
    (dict(oh=60), INV), (dict(os=1784), INV), (dict(os=2308), INV), (dict(out=P((1 << 24) + 8)), INV), (dict(q=P((1 << 22) + 2)), INV),
    # outputs over what is read: the queries shifted, of another pitch, the latent, the key, the pool
    (dict(out=P((1 << 22) + 16), os=768, oh=192), INV), (dict(out=P(1 << 22), os=776, oh=192), INV),
    (dict(out=P(1 << 22), os=2304, oh=576), INV), (dict(out=P(1 << 20)), INV), (dict(out=P((1 << 20) + 1024)), INV),
    (dict(out=P(1 << 50)), INV)])
def test_bad_appends_are_refused(bad, status):
    assert call("kvd_latent_append", append_args(**bad)) == status


@pytest.mark.parametrize("ok", [
    dict(n=0), dict(n=0, latent=None, k=None, slots=None, pos=None, q=None, out=None)])
def test_an_append_of_nothing(ok):
    assert call("kvd_latent_append", append_args(**ok)) == kvd.KVD_OK


def gather_args(**kw):
    a = dict(pool=ctypes.byref(latent()), layer=0, bt=P(4), mb=4, start=P(4), first=None, batch=2, n=3, out=P(16), os=576,
             stream=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(pool=None), INV), (dict(pool=ctypes.byref(fake())), UNS), (dict(layer=2), INV), (dict(batch=-1), INV),
    (dict(n=-1), INV), (dict(mb=0), INV), (dict(batch=2049), UNS), (dict(bt=None), INV), (dict(start=None), INV),
    (dict(out=None), INV), (dict(out=P(8)), INV), (dict(os=568), INV), (dict(os=580), INV), (dict(out=P((1 << 50) + 16)), INV),
    (dict(out=P((1 << 50) - 2304)), INV)])
def test_bad_gathers_are_refused(bad, status):
    assert call("kvd_latent_gather", gather_args(**bad)) == status


def test_a_gather_of_nothing():
    assert call("kvd_latent_gather", gather_args(n=0)) == call("kvd_latent_gather", gather_args(batch=0)) == kvd.KVD_OK


def attn_args(**kw):
    a = dict(pool=ctypes.byref(latent()), layer=0, q=P(1 << 20), n_q=4, start=P(4), n=3, bt=P(4), mb=4, lens=P(4), batch=1,
             retain=None, scale=0.1, ws=P(1 << 30), bytes=1 << 40, out=P(1 << 22), dtype=0, lse=None, stream=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(pool=None), INV), (dict(pool=ctypes.byref(fake())), UNS), (dict(layer=2), INV), (dict(n_q=0), INV),
    (dict(n_q=257), UNS), (dict(batch=-1), INV), (dict(batch=2049), UNS), (dict(n=-1), INV), (dict(mb=0), INV),
    (dict(dtype=1), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(scale=3e38), INV),
    (dict(q=None), INV), (dict(start=None), INV), (dict(bt=None), INV), (dict(lens=None), INV), (dict(ws=None), INV),
    (dict(out=None), INV), (dict(q=P(8)), INV), (dict(out=P(8)), INV), (dict(ws=P(128)), INV), (dict(bytes=1 << 20), MEM),
    (dict(out=P(1 << 20)), INV), (dict(out=P((1 << 20) + 13808)), INV), (dict(out=P(1 << 50)), INV),
    (dict(out=P(1 << 30)), INV), (dict(q=P(1 << 30)), INV)])
def test_bad_attention_is_refused(bad, status):
    assert call("kvd_latent_attn", attn_args(**bad)) == status


def test_attention_over_nothing():
    assert call("kvd_latent_attn", attn_args(n=0)) == call("kvd_latent_attn", attn_args(batch=0)) == kvd.KVD_OK


@pytest.mark.parametrize("n_q,batch,status", [(0, 1, INV), (257, 1, UNS), (4, -1, INV), (4, 2049, UNS)])
def test_workspace_refusals(n_q, batch, status):
    with pytest.raises(kvd.KvdError) as e:
        kvd.kvd_latent_workspace_bytes(ctypes.byref(latent()), n_q, batch)
    assert e.value.status == status


def prefill_args(**kw):
    a = dict(pool=ctypes.byref(latent()), q=P(1 << 20), n_q=4, start=P(4), n=3, k=P(1 << 22), ks=1024, kh=256, v=P((1 << 22) + 256),
             vs=1024, vh=256, r=P(1 << 24), rs=576, kv=P(4), m=5, batch=1, causal=1, scale=0.1, out=P(1 << 26), dtype=0, lse=None,
             stream=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(pool=None), INV), (dict(pool=ctypes.byref(fake())), UNS), (dict(n_q=0), INV), (dict(n_q=257), UNS),
    (dict(batch=-1), INV), (dict(batch=2049), UNS), (dict(n=-1), INV), (dict(m=-1), INV), (dict(causal=2), INV),
    (dict(dtype=3), INV), (dict(scale=float("nan")), INV), (dict(q=None), INV), (dict(start=None), INV), (dict(kv=None), INV),
    (dict(out=None), INV), (dict(q=P(8)), INV), (dict(out=P(8)), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(r=None), INV), (dict(k=P((1 << 22) + 2)), INV), (dict(v=P((1 << 22) + 2)), INV), (dict(r=P(8)), INV),
    (dict(kh=120), INV), (dict(vh=120), INV), (dict(kh=260), INV), (dict(vh=260), INV), (dict(ks=888), INV),
    (dict(vs=888), INV), (dict(ks=1028), INV), (dict(vs=1028), INV), (dict(rs=56), INV), (dict(rs=580), INV),
    (dict(out=P(1 << 20)), INV), (dict(out=P(1 << 22)), INV), (dict(out=P((1 << 22) + 512)), INV), (dict(out=P((1 << 24) + 64)), INV)])
def test_bad_prefills_are_refused(bad, status):
    assert call("kvd_latent_prefill", prefill_args(**bad)) == status


def test_a_prefill_of_nothing():
    assert call("kvd_latent_prefill", prefill_args(n=0)) == call("kvd_latent_prefill", prefill_args(batch=0)) == kvd.KVD_OK


# ------------------------------------------------------------- the Python entry points
@pytest.mark.parametrize("current,dev", [(0, 1), (1, 0), (0, -1)])
@pytest.mark.parametrize("kind", FORMATS + [kvd.KVD_BF16])
def test_a_pools_memory_is_on_the_current_device(monkeypatch, current, dev, kind):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    with pytest.raises(ValueError, match="current device"):
        kvd.kvd_pool_create(1, 1, 4, kind, Tensor((1 << 20,), torch.uint8, dev), d_h=576 if kind in FORMATS else 128)


@pytest.fixture
def library(monkeypatch):
    real = kvd.load()

    class Library:
        def __getattr__(self, name):
            if name in ("kvd_latent_append", "kvd_latent_gather", "kvd_latent_attn", "kvd_latent_prefill"):
                def reached(*_):
                    raise Reached
                return reached
            return getattr(real, name)

    monkeypatch.setattr(kvd._lib, "load", lambda *_: Library())


class View(Tensor):
    def dim(self):
        return len(self.shape)

    def stride(self, dim=None):
        return self.strides if dim is None and hasattr(self, "strides") else \
            self.strides[dim] if hasattr(self, "strides") else super().stride(dim)


def view(shape, dtype, dev=0, strides=None, **kw):
    t = View(shape, dtype, dev, **kw)
    if strides is not None:
        t.strides = strides
    return t


class Rope:
    rot_dim, interleaved, mscale = 64, False, 1.0

    def __init__(self, dev):
        self.turns = Tensor((32, 2), F32, dev)


def append(pool, dev=0, **kw):
    a = dict(latent=view((3, 512), BF16, dev), k_rope=view((3, 64), BF16, dev), slot_mapping=Tensor((3,), I64, dev),
             positions=Tensor((3,), I32, dev), rope=Rope(dev), norm_weight=Tensor((512,), BF16, dev),
             q_rope=view((3, 4, 64), BF16, dev), q_rope_out=view((3, 4, 64), BF16, dev))
    a.update(kw)
    kvd.kvd_latent_append(ctypes.byref(pool), 0, stream=0, **a)


def gather(pool, dev=0, **kw):
    a = dict(block_table=Tensor((2, 4), I32, dev), row_start=Tensor((3,), I32, dev), out=view((9, 576), BF16, dev),
             first=Tensor((2,), I32, dev))
    a.update(kw)
    kvd.kvd_latent_gather(ctypes.byref(pool), 0, stream=0, **a)


def attn(pool, dev=0, **kw):
    a = dict(q=view((3, 4, 576), BF16, dev), q_start=Tensor((2,), I32, dev), block_table=Tensor((1, 4), I32, dev),
             seq_lens=Tensor((1,), I32, dev), workspace=Tensor((1 << 20,), torch.uint8, dev),
             out=view((3, 4, 512), BF16, dev), retain_mask=Tensor((8,), torch.int16, dev), lse_out=Tensor((3, 4), F32, dev))
    a.update(kw)
    kvd.kvd_latent_attn(ctypes.byref(pool), 0, stream=0, **a)


def prefill(pool, dev=0, **kw):
    a = dict(q=view((3, 4, 192), BF16, dev), q_start=Tensor((2,), I32, dev), k_nope=view((5, 4, 128), BF16, dev),
             v=view((5, 4, 128), BF16, dev), k_rope=view((5, 64), BF16, dev), kv_start=Tensor((2,), I32, dev),
             out=view((3, 4, 128), BF16, dev), lse_out=Tensor((3, 4), F32, dev))
    a.update(kw)
    kvd.kvd_latent_prefill(ctypes.byref(pool), stream=0, **a)


CALLS = [append, gather, attn, prefill]


@pytest.mark.parametrize("fn", CALLS)
def test_a_sound_call_passes(library, fn):
    with pytest.raises(Reached):
        fn(latent())


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("pool_device,dev", [(0, -1), (0, 1), (1, 0)])
def test_every_tensor_is_on_the_pools_device(library, fn, pool_device, dev):
    with pytest.raises(ValueError, match="device"):
        fn(latent(device=pool_device), dev=dev)


@pytest.mark.parametrize("fn,bad", [
    (append, dict(latent=view((3, 513), BF16))), (append, dict(latent=view((3, 512), F32))),
    (append, dict(latent=view((3, 512), BF16, strides=(1024, 2)))), (append, dict(k_rope=view((4, 64), BF16))),
    (append, dict(k_rope=view((3, 64), BF16, 1))), (append, dict(slot_mapping=Tensor((3,), I32))),
    (append, dict(slot_mapping=Tensor((2,), I64))), (append, dict(positions=None)), (append, dict(rope=None)),
    (append, dict(positions=Tensor((3,), I64))), (append, dict(rope=Rope(1))), (append, dict(norm_weight=Tensor((512,), F32))),
    (append, dict(norm_weight=Tensor((511,), BF16))), (append, dict(q_rope=view((2, 4, 64), BF16))),
    (append, dict(q_rope=view((3, 4, 63), BF16))), (append, dict(q_rope_out=view((3, 5, 64), BF16))),
    (append, dict(q_rope_out=view((3, 4, 64), BF16, 1))), (append, dict(q_rope=view((3, 4, 64), BF16, strides=(768, 192, 2)))),
    (gather, dict(out=view((9, 512), BF16))), (gather, dict(out=view((9, 576), F32))), (gather, dict(row_start=Tensor((2,), I32))),
    (gather, dict(first=Tensor((3,), I32))), (gather, dict(first=Tensor((2,), I64))), (gather, dict(block_table=Tensor((2, 4), I64))),
    (gather, dict(block_table=Tensor((2, 4), I32, contiguous=False))), (gather, dict(out=view((9, 576), BF16, strides=(1152, 2)))),
    (attn, dict(q=view((3, 4, 512), BF16))), (attn, dict(q=view((3, 4, 576), F32))), (attn, dict(out=view((3, 4, 576), BF16))),
    (attn, dict(out=view((3, 4, 512), torch.float16))), (attn, dict(q=view((3, 4, 576), BF16, contiguous=False))),
    (attn, dict(q_start=Tensor((3,), I32))), (attn, dict(seq_lens=Tensor((1,), I64))), (attn, dict(block_table=Tensor((2, 4), I32))),
    (attn, dict(retain_mask=Tensor((7,), torch.int16))), (attn, dict(retain_mask=Tensor((8,), I32))),
    (attn, dict(workspace=Tensor((1 << 20,), torch.uint8, 1))), (attn, dict(lse_out=Tensor((3, 4), BF16))),
    (attn, dict(lse_out=Tensor((4, 3), F32))),
    (prefill, dict(q=view((3, 4, 128), BF16))), (prefill, dict(k_nope=view((5, 3, 128), BF16))), (prefill, dict(v=view((6, 4, 128), BF16))),
    (prefill, dict(v=view((5, 4, 128), F32))), (prefill, dict(k_rope=view((5, 128), BF16))), (prefill, dict(kv_start=Tensor((3,), I32))),
    (prefill, dict(q_start=Tensor((2,), I64))), (prefill, dict(out=view((3, 4, 192), BF16))), (prefill, dict(out=view((3, 4, 128), torch.float16))),
    (prefill, dict(k_nope=view((5, 4, 128), BF16, strides=(1024, 256, 2)))), (prefill, dict(lse_out=Tensor((3, 5), F32)))])
def test_tensors_of_another_kind(library, fn, bad):
    with pytest.raises(ValueError):
        fn(latent(), **bad)


def test_an_output_without_its_input(library):
    with pytest.raises(ValueError, match="q_rope"):
        append(latent(), q_rope=None)


def test_slices_of_projections_pass(library):
    for a in (dict(latent=view((3, 512), BF16, strides=(576, 1)), k_rope=view((3, 64), BF16, strides=(576, 1)),
                   q_rope=view((3, 4, 64), BF16, strides=(768, 192, 1)), q_rope_out=view((3, 4, 64), BF16, strides=(2304, 576, 1))),
              dict(q_rope=None, q_rope_out=None), dict(q_rope_out=None), dict(norm_weight=None),
              dict(positions=None, rope=None, q_rope=None, q_rope_out=None)):
        with pytest.raises(Reached):
            append(latent(), **a)
    with pytest.raises(Reached):
        prefill(latent(), k_nope=view((5, 4, 128), BF16, strides=(1024, 256, 1)), v=view((5, 4, 128), BF16, strides=(1024, 256, 1)),
                k_rope=view((5, 64), BF16, strides=(576, 1)), lse_out=None, causal=False)
    with pytest.raises(Reached):
        gather(latent(), first=None, out=view((9, 576), BF16, strides=(640, 1)))
