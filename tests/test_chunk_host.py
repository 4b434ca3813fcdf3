"""Host side of the chunk operators: the rotary rules against their formulas, and every refusal."""

import ctypes
import math

import numpy as np
import pytest

import paged_gqa_decode_kvd_gb300 as kvd
from chunk_ref import rope_freqs_ref

INV, UNS, MEM = kvd.KVD_ERR_INVALID, kvd.KVD_ERR_UNSUPPORTED, kvd.KVD_ERR_NOMEM
P = ctypes.c_void_p


@pytest.mark.parametrize("rule", [{}, dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                  dict(scaling="banded", factor=8.0, original_len=8192, low=1.0, high=4.0),
                                  dict(scaling="yarn", factor=40.0, original_len=4096, low=1.0, high=32.0)])
@pytest.mark.parametrize("rot,base", [(128, 500000.0), (64, 10000.0), (66, 1e6), (4, 10000.0)])
def test_frequencies_follow_the_rules(rule, rot, base):
    turns, m = kvd.kvd_rope_freqs(rot, base, **rule)
    theta, want_m = rope_freqs_ref(rot, base, **rule)
    got = turns.astype(np.float64).sum(1) * 2 * math.pi
    # two floats hold 48 bits; the formulas in fp64 differ by a few of its roundings (pow: relative |log| ulp)
    assert np.abs(got / theta - 1).max() < 2.0 ** -44
    assert m == np.float32(want_m)
    assert (np.abs(turns[:, 1]) <= np.abs(turns[:, 0]) * 2.0 ** -24).all()


@pytest.mark.parametrize("bad,status", [
    (dict(rot_dim=3), INV), (dict(rot_dim=0), INV), (dict(rot_dim=130), UNS), (dict(base=1.0), INV),
    (dict(base=float("nan")), INV), (dict(base=float("inf")), INV), (dict(scaling="linear", factor=0.5), INV),
    (dict(scaling="ntk", factor=2.0, rot_dim=2), INV), (dict(scaling="ntk", factor=float("nan")), INV),
    (dict(scaling="banded", factor=2.0, original_len=0, low=1, high=4), INV),
    (dict(scaling="banded", factor=2.0, original_len=8192, low=4, high=4), INV),
    (dict(scaling="yarn", factor=2.0, original_len=8192, low=0, high=4), INV),
    (dict(scaling="yarn", factor=float("inf"), original_len=8192, low=1, high=4), INV)])
def test_bad_rules_are_refused(bad, status):
    with pytest.raises(kvd.KvdError) as e:
        kvd.kvd_rope_freqs(**{**dict(rot_dim=64, base=10000.0), **bad})
    assert e.value.status == status


def test_unknown_rule_is_refused():
    with pytest.raises(ValueError):
        kvd.kvd_rope_freqs(64, 10000.0, scaling="other")
    sc = kvd._lib.RopeScaling(5, 1.0, 1.0, 1.0, 2.0)
    buf = np.zeros(64, np.float32)
    assert kvd.load().kvd_rope_freqs(64, 10000.0, ctypes.byref(sc), buf.ctypes.data_as(P),
                                     ctypes.byref(ctypes.c_float())) == INV


class FakePool(ctypes.Structure):
    """The fields a check reads, laid out as the library's handle: no call here gets as far as a launch."""
    _fields_ = [("desc", kvd._lib.PoolDesc), ("mem", P), ("err", P), ("device", ctypes.c_int),
                ("num_sms", ctypes.c_int), ("layer_bytes", ctypes.c_size_t), ("host_kv", P), ("host_mem", P),
                ("staging", P), ("host_blocks", ctypes.c_int64), ("host_layer_bytes", ctypes.c_size_t),
                ("host_direct", ctypes.c_int), ("block_fmt", P), ("block_fmt_count", ctypes.c_int64)]


def fake(kind=kvd.KVD_BF16, n_kv=2, blocks=8, layers=2):
    f = FakePool()
    f.desc = kvd._lib.PoolDesc(layers, n_kv, 128, 16, blocks, kind, 32)
    f.num_sms = 152
    return f


def rope_args(handle, **kw):
    d = kvd._lib.RopeDesc(4096, 128, 0, 1.0)
    a = dict(pool=ctypes.byref(handle), layer=0, q=P(16), qs=512, n_q=4, k=P(16), ks=256, v=P(16), vs=256, pos=P(4),
             rope=d, slots=P(8), n=3, q_out=P(32), os=512)
    a.update(kw)
    for k in ("rot", "inter", "turns"):
        if k in kw:
            setattr(d, {"rot": "rot_dim", "inter": "interleaved", "turns": "turns"}[k], a.pop(k))
    r = a["rope"]
    return (a["pool"], a["layer"], a["q"], a["qs"], a["n_q"], a["k"], a["ks"], a["v"], a["vs"], a["pos"],
            None if r is None else ctypes.byref(r), a["slots"], a["n"], a["q_out"], a["os"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(pool=None), INV), (dict(layer=2), INV), (dict(layer=-1), INV), (dict(n_q=-1), INV), (dict(n=-1), INV),
    (dict(rope=None), INV), (dict(rot=3), INV), (dict(rot=0), INV), (dict(rot=130), UNS), (dict(inter=2), INV),
    (dict(turns=None), INV), (dict(turns=4100), INV), (dict(q=None), INV), (dict(q_out=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(pos=None), INV), (dict(slots=None), INV), (dict(ks=248), INV), (dict(vs=260), INV),
    (dict(qs=504), INV), (dict(qs=516), INV), (dict(os=500), INV), (dict(q=P(8)), INV), (dict(k=P(8)), INV),
    (dict(v=P(24)), INV), (dict(q_out=P(40)), INV), (dict(q_out=P(16), os=1024), INV), (dict(n_q=65537, qs=1 << 24), UNS),
    (dict(n=0), kvd.KVD_OK), (dict(n=0, k=None, v=None, pos=None, slots=None), kvd.KVD_OK)])
def test_rope_append_refusals(kw, status):
    assert kvd.load().kvd_rope_append(*rope_args(fake(), **kw)) == status


def test_rope_append_needs_the_formats_of_a_mixed_pool():
    assert kvd.load().kvd_rope_append(*rope_args(fake(kvd.KVD_MIXED))) == INV


@pytest.mark.parametrize("kw,status", [
    (dict(pool=None), INV), (dict(layer=2), INV), (dict(n_q=0), INV), (dict(n_q=3), INV), (dict(n_q=18), UNS),
    (dict(batch=-1), INV), (dict(batch=2049), UNS), (dict(n=-1), INV), (dict(mb=0), INV), (dict(dt=kvd.KVD_MIXED), INV),
    (dict(q=None), INV), (dict(q=P(8)), INV), (dict(start=None), INV), (dict(bt=None), INV), (dict(lens=None), INV),
    (dict(ws=None), INV), (dict(ws=P(128)), INV), (dict(wb=0), MEM), (dict(out=None), INV), (dict(out=P(24)), INV),
    (dict(batch=0), kvd.KVD_OK), (dict(n=0), kvd.KVD_OK), (dict(n=0, q=None, out=None, ws=None), kvd.KVD_OK)])
def test_chunk_attn_refusals(kw, status):
    a = dict(pool=ctypes.byref(fake()), layer=0, q=P(16), n_q=4, start=P(4), n=3, bt=P(4), mb=4, lens=P(4), batch=1,
             ws=P(256), wb=1 << 40, out=P(16), dt=kvd.KVD_BF16)
    a.update(kw)
    assert kvd.load().kvd_chunk_attn(a["pool"], a["layer"], a["q"], a["n_q"], a["start"], a["n"], a["bt"], a["mb"],
                                     a["lens"], a["batch"], None, 0.1, a["ws"], a["wb"], a["out"], a["dt"], None,
                                     None) == status


def test_chunk_attn_needs_the_formats_of_a_mixed_pool():
    f = fake(kvd.KVD_MIXED)
    assert kvd.load().kvd_chunk_attn(ctypes.byref(f), 0, P(16), 4, P(4), 3, P(4), 4, P(4), 1, None, 0.1, P(256), 1 << 40,
                                     P(16), kvd.KVD_BF16, None, None) == INV
    n = ctypes.c_size_t()
    assert kvd.load().kvd_chunk_workspace_bytes(ctypes.byref(fake()), 4, 1, None) == INV
    assert kvd.load().kvd_chunk_workspace_bytes(ctypes.byref(fake()), 4, 1, ctypes.byref(n)) == kvd.KVD_OK and n.value > 0


@pytest.mark.parametrize("kw,status", [
    (dict(pool=None), INV), (dict(batch=-1), INV), (dict(batch=65536), UNS), (dict(mb=0), INV), (dict(nmb=0), INV),
    (dict(bt=None), INV), (dict(lens=None), INV), (dict(new=None), INV), (dict(nl=None), INV), (dict(nl=P(64)), INV),
    (dict(ws=None), INV), (dict(ws=P(16)), INV), (dict(wb=16), MEM), (dict(sc=P(4)), INV), (dict(nsc=P(4)), INV),
    (dict(sc=P(4), nsc=P(4)), INV), (dict(sc=P(4), nsc=P(8), ss=0), INV), (dict(sc=P(4), nsc=P(8), ns=0), INV),
    (dict(batch=0), kvd.KVD_OK)])
def test_compact_refusals(kw, status):
    a = dict(pool=ctypes.byref(fake()), bt=P(4), mb=4, lens=P(64), batch=2, new=P(4), nmb=4, nl=P(128), sc=None, ss=8,
             nsc=None, ns=8, ws=P(256), wb=1 << 20)
    a.update(kw)
    assert kvd.load().kvd_compact(a["pool"], a["bt"], a["mb"], a["lens"], a["batch"], None, a["new"], a["nmb"], a["nl"],
                                  a["sc"], a["ss"], a["nsc"], a["ns"], a["ws"], a["wb"], None) == status


def test_compact_pools_that_cannot():
    n = ctypes.c_size_t()
    lib = kvd.load()
    assert lib.kvd_compact_workspace_bytes(ctypes.byref(fake(kvd.KVD_MIXED)), 1, 4, ctypes.byref(n)) == UNS
    assert lib.kvd_compact_workspace_bytes(ctypes.byref(fake(blocks=(1 << 27) + 1)), 1, 4, ctypes.byref(n)) == UNS
    assert lib.kvd_compact_workspace_bytes(ctypes.byref(fake()), 1, 4, None) == INV
    assert lib.kvd_compact_workspace_bytes(ctypes.byref(fake()), 3, 5, ctypes.byref(n)) == kvd.KVD_OK
    assert n.value >= 3 * 5 * 16 * 4 + 8 * 4
