"""GPU tests of the rotary and block-sparse calls at the ends of their ranges: a
batch without tokens, key bounds beyond 32-bit offsets."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_key_bounds_beyond_32_bits(pa, dtype):
    """Bounds whose own offsets pass 2^32 elements (fp32: 2^31), written and
    scored at the far end as at the near one."""
    hkv, bs, d = 8, 8, 128
    NB = ((1 << 32) if dtype == torch.bfloat16 else (1 << 31)) // (hkv * 2 * d) + 9
    # 34 GB of keys; only the used blocks are written
    kp = torch.empty(NB, hkv, bs, d, dtype=dtype, device="cuda")
    kb = torch.empty(NB, hkv, 2, d, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    keys = torch.randn(3, hkv, bs, d, generator=g, device="cuda").to(dtype)
    q = torch.randn(1, 2 * hkv, d, generator=g, device="cuda").to(dtype)
    near, far = [2, 0, 1], [NB - 1, NB // 2 + 1, NB - 7]
    got = []
    for blocks in (far, near):
        at = torch.tensor(blocks, device="cuda")
        kp[at], kb[at] = keys, 0
        lens, tables = i32([2 * bs + 5]), i32([blocks])
        pa.pa_update_key_bounds(kp, kb, tables, lens, query_start=i32([0, 2 * bs + 5]), max_query_len=2 * bs + 5)
        scores = torch.full((1, hkv, 3), -7.0, device="cuda")
        pa.pa_block_scores(q, kb, tables, lens, 2 * bs + 5, bs, scores)
        assert torch.equal(kb[at][:2], torch.stack([keys[:2].amin(2), keys[:2].amax(2)], 2))
        assert torch.equal(kb[at][2], torch.stack([keys[2, :, :5].amin(1), keys[2, :, :5].amax(1)], 1))
        got.append(scores)
    assert torch.equal(*got) and (got[0] != -7).all()
    assert pa.pa_read_error_flag() == 0
