"""Refusals of the chunk operators that need a device."""

import ctypes

import pytest
import torch

import paged_gqa_decode_kvd_gb300 as kvd
from test_chunk_checks import chunk, compact, handle, rope
from test_chunk_host import P, fake, rope_args

pytestmark = pytest.mark.gpu


def test_another_current_device_is_refused(cuda_device):
    """A pool whose device is not the current one: refused before a launch (a kernel would run beside its memory)."""
    torch.cuda.current_stream()
    pool = fake()
    pool.device = torch.cuda.current_device() + 1
    lib = kvd.load()
    assert lib.kvd_rope_append(*rope_args(pool)) == kvd.KVD_ERR_INVALID
    assert lib.kvd_chunk_attn(ctypes.byref(pool), 0, P(16), 4, P(4), 3, P(4), 4, P(4), 1, None, 0.1, P(256), 1 << 40,
                              P(1 << 20), kvd.KVD_BF16, None, None) == kvd.KVD_ERR_INVALID
    assert lib.kvd_compact(ctypes.byref(pool), P(4), 4, P(64), 2, None, P(4), 4, P(128), None, 8, None, 8, P(256), 1 << 20,
                           None) == kvd.KVD_ERR_INVALID
    for call in (chunk, compact, rope):
        with pytest.raises(ValueError):
            call(handle(device=pool.device))
