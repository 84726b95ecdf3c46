"""GPU tests of the rotary and block-sparse calls at the ends of their ranges: a
batch without tokens."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_355_b200 as pa

    assert torch.cuda.is_available()
    pa.pa_read_error_flag()  # clear
    return pa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_a_step_of_empty_sequences(pa):
    """Padding rows only: nothing written, nothing scored, no block chosen, zeros."""
    B, hq, hkv, d, bs = 3, 4, 2, 64, 16
    qkv = torch.randn(B, hq + 2 * hkv, d, device="cuda")
    kp, vp = torch.randn(5, hkv, bs, d, device="cuda"), torch.randn(5, hkv, bs, d, device="cuda")
    kb, before = torch.randn(5, hkv, 2, d, device="cuda"), (kp.clone(), vp.clone())
    bounds = kb.clone()
    query_out = torch.full((B, hq, d), 7.0, device="cuda")
    scores = torch.zeros(B, hkv, 0, device="cuda")
    selected = torch.full((B, hkv, 3), 9, dtype=torch.int32, device="cuda")
    out = torch.full((B, hq, d), 7.0, device="cuda")
    slots = torch.full((B,), 5, dtype=torch.int64, device="cuda")
    pa.sparse_decode_step(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp, kb, i32([[0], [1], [-1]]),
                          i32([0, 0, 0]), 0, torch.ones(1, d, device="cuda"), 0.125, query_out, scores, selected, out,
                          slots=slots)
    assert (query_out == 7).all() and (slots == -1).all() and (selected == -1).all() and not out.any()
    assert torch.equal(kp, before[0]) and torch.equal(vp, before[1]) and torch.equal(kb, bounds)
    assert pa.pa_read_error_flag() == 0
    # a length that the empty scores cannot hold is flagged, not read
    pa.pa_select_blocks(scores, i32([0, 1, 0]), 0, bs, selected.fill_(9))
    assert (selected == -1).all() and pa.pa_read_error_flag() == 5
