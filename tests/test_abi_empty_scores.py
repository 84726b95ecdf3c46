"""A batch without tokens: no score columns, so no score array.  No GPU: the
call gets past its checks and fails only where it needs a device."""
from __future__ import annotations

import ctypes

import pytest
import torch

INVALID, CUDA = 1, 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are no device memory")
def test_selection_takes_scores_without_columns():
    from paged_kv_cache_355_b200 import build

    lib = ctypes.CDLL(build.build())
    P, I64 = ctypes.c_void_p, ctypes.c_int64
    call = lambda scores, stride, longest: lib.pa_select_blocks(P(scores), I64(stride), P(16), longest, 16, P(16), 4, 1, 2,
                                                                I64(2), 2, None)
    assert call(0, 0, 0) == CUDA
    assert call(0, 1, 0) == INVALID   # columns, and no address
    assert call(0, 0, 1) == INVALID   # a block, and no column for it
