"""What the Python entry points of the chunk operators refuse before the library sees it: tensors of another device,
type or size than the pool's.  Tensors are stand-ins with the attributes a check reads; nothing is launched."""

import ctypes

import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from test_chunk_host import fake, rope_args

BF16, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


class Tensor:
    """A contiguous device tensor, as far as a check can tell."""

    def __init__(self, shape, dtype, device=0, contiguous=True, at=4096):
        self.shape, self.dtype, self.device_index, self.contiguous, self.at = torch.Size(shape), dtype, device, contiguous, at

    def stride(self, dim=None):
        s = torch.empty(self.shape, device="meta").stride()
        return s if dim is None else s[dim]

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    def data_ptr(self):
        return self.at


class Reached(Exception):
    pass


@pytest.fixture
def library(monkeypatch):
    """The library with its launching entry points replaced: a call that passes the checks raises Reached."""
    real = kvd.load()

    class Library:
        def __getattr__(self, name):
            if name in ("kvd_chunk_attn", "kvd_compact", "kvd_rope_append"):
                def reached(*_):
                    raise Reached
                return reached
            return getattr(real, name)

    monkeypatch.setattr(kvd._lib, "load", lambda *_: Library())


def handle(device=0, host_blocks=0, **kw):
    f = fake(**kw)
    f.device, f.host_blocks = device, host_blocks
    return f


def chunk(pool, dev=0, **kw):
    a = dict(q=Tensor((3, 4, 128), BF16, dev), q_start=Tensor((2,), I32, dev), block_table=Tensor((1, 4), I32, dev),
             seq_lens=Tensor((1,), I32, dev), workspace=Tensor((1 << 20,), torch.uint8, dev),
             out=Tensor((3, 4, 128), BF16, dev), retain_mask=Tensor((8,), torch.int16, dev),
             lse_out=Tensor((3, 4), F32, dev))
    a.update(kw)
    kvd.kvd_chunk_attn(ctypes.byref(pool), 0, stream=0, **a)


def compact(pool, dev=0, **kw):
    a = dict(block_table=Tensor((2, 4), I32, dev), seq_lens=Tensor((2,), I32, dev), new_table=Tensor((2, 4), I32, dev),
             new_lens=Tensor((2,), I32, dev, at=8192), workspace=Tensor((1 << 20,), torch.uint8, dev),
             retain_mask=Tensor((8,), torch.int16, dev), scores=Tensor((2, 64), F32, dev),
             new_scores=Tensor((2, 64), F32, dev, at=8192))
    a.update(kw)
    kvd.kvd_compact(ctypes.byref(pool), stream=0, **a)


class Rope:
    rot_dim, interleaved, mscale = 128, False, 1.0

    def __init__(self, dev):
        self.turns = Tensor((64, 2), F32, dev)


def rope(pool, dev=0, **kw):
    a = dict(q=Tensor((3, 4, 128), BF16, dev), k_new=Tensor((3, 2, 128), BF16, dev), v_new=Tensor((3, 2, 128), BF16, dev),
             positions=Tensor((3,), I32, dev), rope=Rope(dev), slot_mapping=Tensor((3,), I64, dev),
             q_out=Tensor((3, 4, 128), BF16, dev))
    a.update(kw)
    kvd.kvd_rope_append(ctypes.byref(pool), 0, stream=0, **a)


@pytest.mark.parametrize("call", [chunk, compact, rope])
def test_a_sound_call_passes(library, call):
    with pytest.raises(Reached):
        call(handle())


@pytest.mark.parametrize("call", [chunk, compact, rope])
@pytest.mark.parametrize("pool_device,dev", [(0, -1), (0, 1), (1, 0)])
def test_every_tensor_is_on_the_pools_device(library, call, pool_device, dev):
    """-1 is host memory: all tensors there agree with each other, and the kernels cannot read them."""
    with pytest.raises(ValueError, match="device"):
        call(handle(device=pool_device), dev=dev)


@pytest.mark.parametrize("call", [chunk, compact])
def test_the_mask_covers_the_pool(library, call):
    """Block ids run over the pool's and the host tier's blocks; compaction writes the mask of a new block."""
    for blocks, host in ((8, 0), (8, 5), (1000, 0)):
        pool = handle(blocks=blocks, host_blocks=host)
        with pytest.raises(Reached):
            call(pool, retain_mask=Tensor((blocks + host,), torch.int16))
        with pytest.raises(Reached):
            call(pool, retain_mask=Tensor((blocks + host,), torch.uint16))
        with pytest.raises(Reached):
            call(pool, retain_mask=None)
        with pytest.raises(ValueError, match="retain_mask"):
            call(pool, retain_mask=Tensor((blocks + host - 1,), torch.int16))


@pytest.mark.parametrize("call", [chunk, compact])
@pytest.mark.parametrize("mask", [Tensor((8,), torch.int32), Tensor((8,), torch.uint8), Tensor((8,), torch.bool),
                                  Tensor((8,), torch.int16, device=-1), Tensor((8,), torch.int16, device=1),
                                  Tensor((8,), torch.int16, contiguous=False)])
def test_masks_of_another_kind(library, call, mask):
    with pytest.raises(ValueError, match="retain_mask"):
        call(handle(), retain_mask=mask)


@pytest.mark.parametrize("call", [chunk, compact])
@pytest.mark.parametrize("workspace", [Tensor((1 << 20,), torch.uint8, device=-1), Tensor((1 << 20,), torch.uint8, device=1),
                                       Tensor((1 << 20,), torch.uint8, contiguous=False)])
def test_workspaces_elsewhere(library, call, workspace):
    with pytest.raises(ValueError, match="workspace"):
        call(handle(), workspace=workspace)


class Wide(Tensor):
    """A slice of a projection's output, 512 heads wide."""

    def stride(self, dim=None):
        s = (512 * 128, 128, 1)
        return s if dim is None else s[dim]


@pytest.mark.parametrize("kind", [Tensor, Wide])
@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_keys_have_the_pools_heads(library, kind, tokens, heads):
    """The kernel reads the pool's two heads from every token's row: with fewer it would read past the slice, with more
    the others would be lost."""
    kv = dict(k_new=kind((tokens, heads, 128), BF16), v_new=kind((tokens, heads, 128), BF16), q=None, q_out=None,
              positions=Tensor((tokens,), I32), slot_mapping=Tensor((tokens,), I64))
    with pytest.raises(ValueError, match="heads"):
        rope(handle(), **kv)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_a_scale_that_is_no_number_is_refused(scale):
    """A NaN became the smallest scale, and every position weighed the same."""
    p = ctypes.c_void_p
    assert kvd.load().kvd_chunk_attn(ctypes.byref(fake()), 0, p(16), 4, p(4), 3, p(4), 4, p(4), 1, None, scale, p(256),
                                     1 << 40, p(1 << 20), kvd.KVD_BF16, None, None) == kvd.KVD_ERR_INVALID


@pytest.mark.parametrize("dtype,distance", [(kvd.KVD_BF16, 0), (kvd.KVD_BF16, 5104), (kvd.KVD_BF16, -5104),
                                            (kvd.KVD_F32, 5104), (kvd.KVD_F32, -10224)])
def test_out_over_q_is_refused(dtype, distance):
    """Five tokens of four heads: 5,120 bytes of q, as many of out or twice that.  16 bytes further they are apart: such a
    call gets as far as the device check, which a pool of a device that is not there does not pass."""
    p, pool = ctypes.c_void_p, handle(device=99)

    def call(at):
        return kvd.load().kvd_chunk_attn(ctypes.byref(pool), 0, p(1 << 20), 4, p(4), 5, p(4), 4, p(4), 1, None, 0.1, p(256),
                                         1 << 40, p((1 << 20) + at), dtype, None, None)

    assert call(distance) == kvd.KVD_ERR_INVALID
    if distance and not torch.cuda.is_available():
        assert call(distance + (16 if distance > 0 else -16)) == kvd.KVD_ERR_CUDA


def status_of_rope(q_out, os=512, q=1 << 20, qs=1024, k=(1 << 20) + 1024, v=(1 << 20) + 1536, n=5):
    """Five tokens of one projection, a row of 2,048 bytes: four query heads, two key heads, two value heads."""
    p, pool = ctypes.c_void_p, handle(device=99)
    return kvd.load().kvd_rope_append(*rope_args(pool, q=p(q), qs=qs, k=p(k), ks=1024, v=p(v), vs=1024, n=n, q_out=p(q_out),
                                                 os=os))


APART = kvd.KVD_ERR_INVALID if torch.cuda.is_available() else kvd.KVD_ERR_CUDA   # as far as the device check


@pytest.mark.parametrize("q_out,stride", [(1 << 20, 512), ((1 << 20) + 16, 1024), ((1 << 20) - 16, 1024),
                                          ((1 << 20) + 1008, 1024), ((1 << 20) + 1024, 1024), ((1 << 20) + 2048 - 16, 1024),
                                          ((1 << 20) + 2048, 1024), ((1 << 20) + 1536, 512), ((1 << 20) - 5104, 512)])
def test_rotated_queries_over_the_inputs_are_refused(q_out, stride):
    assert status_of_rope(q_out, stride) == kvd.KVD_ERR_INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="tells a refusal from the device check by the lack of a device")
def test_rotated_queries_apart_from_the_inputs_pass():
    assert status_of_rope(1 << 20, 1024) == APART                    # q itself
    assert status_of_rope(1 << 22, 512) == APART                     # a tensor of its own
    assert status_of_rope(1 << 20, 1024, k=1 << 20) == APART         # keys rotated in place, without slots
    assert status_of_rope(1 << 20, 1024, k=1 << 20, v=1 << 20) == APART
    assert status_of_rope((1 << 20) - 5120, 512) == APART            # right before the projection
    # the unused part of a wider projection (a row of 4,096 bytes)
    p, pool = ctypes.c_void_p, handle(device=99)
    args = dict(q=p(1 << 20), qs=2048, k=p((1 << 20) + 1024), ks=2048, v=p((1 << 20) + 1536), vs=2048, n=5, os=2048)
    for at, want in ((2048, APART), (2560, APART), (4096 - 1008, kvd.KVD_ERR_INVALID), (2032, kvd.KVD_ERR_INVALID)):
        assert kvd.load().kvd_rope_append(*rope_args(pool, q_out=p((1 << 20) + at), **args)) == want


@pytest.mark.parametrize("lens,new_lens,scores,new_scores", [
    (4096, 4096 + 4, None, None), (4096 + 4, 4096, None, None), (4096, 8192, 16384, 16384 + 4),
    (4096, 8192, 16384 + 508, 16384), (4096, 8192, 16384, 16384 + 508)])
def test_compaction_writes_over_nothing_it_reads(lens, new_lens, scores, new_scores):
    """Two requests, 64 scores each: 8 bytes of lengths, 512 of scores."""
    p, pool = ctypes.c_void_p, handle(device=99)
    assert kvd.load().kvd_compact(ctypes.byref(pool), p(64), 4, p(lens), 2, None, p(128), 4, p(new_lens),
                                  p(scores), 64, p(new_scores), 64, p(256), 1 << 20, None) == kvd.KVD_ERR_INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="tells a refusal from the device check by the lack of a device")
def test_compaction_apart_passes():
    p, pool = ctypes.c_void_p, handle(device=99)
    assert kvd.load().kvd_compact(ctypes.byref(pool), p(64), 4, p(4096), 2, None, p(128), 4, p(4096 + 8), p(16384), 64,
                                  p(16384 + 512), 64, p(256), 1 << 20, None) == kvd.KVD_ERR_CUDA


def test_pool_info():
    desc, host, device = kvd.kvd_pool_info(ctypes.byref(handle(device=3, host_blocks=7, n_kv=4, blocks=9)))
    assert (desc.n_kv, desc.num_blocks, host, device) == (4, 9, 7, 3)
    with pytest.raises(kvd.KvdError):
        kvd.kvd_pool_info(None)
