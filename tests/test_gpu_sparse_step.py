"""GPU tests of sparse_decode_step's other arguments: copy-on-write pairs, and
rotary positions of several axes, each stage against its fp64 definition."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import rope_sparse as rs
from tests.helpers import assert_matches_oracle, np_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_355_b200 as pa

    assert torch.cuda.is_available()
    pa.pa_read_error_flag()  # clear
    return pa


def f64(t):
    return t.detach().cpu().double().numpy()


HQ, HKV, D, K = 8, 2, 64, 4


def angles(last, rotary):
    freq = 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) * 2 / rotary)
    a = torch.arange(last, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def step_and_check(pa, qkv, kp, vp, kb, tables, lens, bs, cos_sin, first, last, slots, **kw):
    """One step on the GPU; every stage's result against its definition on the
    GPU's own inputs to that stage.  `slots`: what the new tokens' slots have to
    be.  Returns the rotated queries."""
    B, longest, scale = qkv.shape[0], max(lens), float(np.float32(1 / math.sqrt(D)))
    blocks = -(-longest // bs)
    out, query_out = torch.zeros(B, HQ, D, device="cuda"), torch.zeros(B, HQ, D, dtype=qkv.dtype, device="cuda")
    scores = torch.zeros(B, HKV, blocks, device="cuda")
    selected = torch.zeros(B, HKV, K, dtype=torch.int32, device="cuda")
    got_slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    p = qkv.cuda()
    pa.sparse_decode_step(p[:, :HQ], p[:, HQ:HQ + HKV], p[:, HQ + HKV:], kp, vp, kb, torch.tensor(tables, dtype=torch.int32).cuda(),
                          torch.tensor(lens, dtype=torch.int32).cuda(), longest, cos_sin.cuda(), scale, query_out, scores,
                          selected, out, slots=got_slots, num_first=first, num_last=last, **kw)
    assert pa.pa_read_error_flag() == 0 and got_slots.tolist() == list(slots)
    want = np.zeros_like(f64(scores))
    size = rs.block_scores(f64(query_out), f64(kb), tables, range(B), lens, bs, want)
    assert (np.abs(f64(scores) - want) <= (2 * D + 2) * 2.0 ** -23 * size).all()
    chosen = rs.select_blocks(scores.cpu().numpy(), lens, bs, K, first, last)
    assert np.array_equal(selected.cpu().numpy(), chosen)
    assert_matches_oracle(out, rs.sparse_decode(f64(query_out), f64(kp), f64(vp), tables, range(B), lens, chosen.tolist(), scale),
                          qkv.dtype == torch.bfloat16)
    return query_out


def check_write(qkv, kp0, vp0, query_out, kp, vp, slots, positions, cos_sin, pair_axes, interleaved, half_step):
    """The queries and both whole pools after the write, from the pools before it."""
    want_q, want_k, want_v, x = np.zeros(query_out.shape), f64(kp0), f64(vp0), f64(qkv)
    qs, ks = rs.rope_and_cache(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], slots, positions, f64(cos_sin), pair_axes,
                               interleaved, None, None, 1e-6, want_q, want_k, want_v)
    for got, ref, size in ((query_out, want_q, qs), (kp, want_k, ks)):
        bound = np.where(size > 0, half_step * np.abs(ref) + 16 * 2.0 ** -24 * size, 0.0) * (1 + 2.0 ** -7)
        assert (np.abs(f64(got) - ref) <= bound).all()
    assert np.array_equal(f64(vp), want_v)


@pytest.mark.parametrize("bs,prompt", [(8, 37), (16, 41)])
def test_copy_on_write(pa, bs, prompt):
    """Three samples share a prompt whose last block is filled in part, and a
    fourth sequence stands alone.  At the first step the block manager hands out
    copies of that block: the copies get the bounds of the tokens they then hold,
    and the block that is left to the last sharer its own, at every step."""
    from paged_kv_cache_355_b200.block_manager import BlockManager

    g = torch.Generator().manual_seed(bs)
    draw = lambda *s: torch.randn(*s, generator=g).bfloat16()
    NB = 40
    kp, vp = draw(NB, HKV, bs, D).cuda(), draw(NB, HKV, bs, D).cuda()
    kb = draw(NB, HKV, 2, D).cuda()
    bm = BlockManager(NB, bs)
    bm.append_tokens([0] * prompt)
    bm.append_tokens([3] * (bs + 3))
    for child in (1, 2):
        bm.fork(0, child)
    tables, lens = bm.block_tables([0, 3], 8)
    starts = torch.tensor([0, lens[0], lens.sum()], dtype=torch.int32).cuda()
    pa.pa_update_key_bounds(kp, kb, torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), query_start=starts,
                            max_query_len=int(lens.max()))
    cos_sin, copies = angles(100, D), 0
    for step in range(3):
        slots, pairs = bm.append_tokens([0, 1, 2, 3])
        copies += len(pairs)
        tables, lens = bm.block_tables([0, 1, 2, 3], 8)
        tables, lens = tables.tolist(), lens.tolist()
        hk, hv, hb = np_of(kp).copy(), np_of(vp).copy(), f64(kb)
        oracle.copy_blocks(hk, hv, pairs)
        to_bf16 = lambda bits: torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
        kp0, vp0 = to_bf16(hk), to_bf16(hv)
        qkv = draw(4, HQ + 2 * HKV, D)
        query_out = step_and_check(pa, qkv, kp, vp, kb, tables, lens, bs, cos_sin, 1, 2, slots,
                                   cow_pairs=torch.from_numpy(pairs).cuda())
        check_write(qkv, kp0, vp0, query_out, kp, vp, slots, np.array([lens]) - 1, cos_sin, None, False, 2.0 ** -8)
        # the running bounds are those of all tokens held, and no other block's moved
        rs.update_key_bounds(f64(kp), hb, tables, lens, [1] * 4)
        assert np.array_equal(f64(kb), hb)
        rs.update_key_bounds(f64(kp), hb, tables, lens, lens)
        assert np.array_equal(f64(kb), hb)
    assert copies == 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("first,last", [(0, 1), (2, 0), (3, 1)])
def test_several_axes_and_other_fixed_blocks(pa, dtype, interleaved, first, last):
    from paged_kv_cache_355_b200.workloads import custom_case

    bs, rotary, lens = 16, 48, [130, 17, 300, 1]
    case = custom_case(lens, HQ, HKV, D, bs, dtype, seed=3)
    g = torch.Generator().manual_seed(first)
    tables = case.block_tables.tolist()
    kp, vp = case.k_pool.cuda(), case.v_pool.cuda()
    kb = torch.zeros(case.num_blocks, HKV, 2, D, dtype=dtype, device="cuda")
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    pa.pa_update_key_bounds(kp, kb, case.block_tables.cuda(), case.lengths.cuda(), query_start=starts, max_query_len=300)
    qkv = torch.randn(4, HQ + 2 * HKV, D, generator=g).to(dtype)
    positions = torch.randint(0, 90, (3, 4), generator=g, dtype=torch.int32)
    pair_axes = torch.randint(0, 3, (rotary // 2,), generator=g, dtype=torch.int32)
    slots = [tables[b][(L - 1) // bs] * bs + (L - 1) % bs for b, L in enumerate(lens)]
    cos_sin = angles(90, rotary)
    query_out = step_and_check(pa, qkv, kp, vp, kb, tables, lens, bs, cos_sin, first, last, slots,
                               positions=positions.cuda(), pair_axes=pair_axes.cuda(), interleaved=interleaved)
    check_write(qkv, case.k_pool, case.v_pool, query_out, kp, vp, slots, positions.numpy(), cos_sin, pair_axes.numpy(),
                interleaved, 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8)
    bounds = f64(kb)
    rs.update_key_bounds(f64(kp), bounds, tables, lens, lens)
    assert np.array_equal(f64(kb), bounds)
