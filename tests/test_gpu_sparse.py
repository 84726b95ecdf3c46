"""GPU parity of block-sparse decode (key bounds, block scores, selection,
attention over the selected blocks) against the fp64 definitions.

Bounds and selections are exact.  A score is a sum of 2 * head_dim products
that are exact in fp32 for bf16 inputs (one more rounding each for fp32), each
addition off by at most one step 2^-23 of a partial sum, so by
(2 D + 2) 2^-23 sum|terms| in all.  Attention is held to the bars of the dense
decode tests: 1e-5 for fp32, 2e-3 (and 1e-2 relative) for bf16 inputs with
fp32 output, one bf16 step for bf16 output.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import rope_sparse as rs
from paged_kv_cache_355_b200.workloads import custom_case
from tests.helpers import assert_matches_oracle, np_of

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_355_b200 as pa

    assert torch.cuda.is_available()
    pa.pa_read_error_flag()  # clear
    return pa


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ---------------------------------------------------------------------------
# key bounds
# ---------------------------------------------------------------------------
def poison_past_lengths(case, value=float("nan")):
    """Every pool slot that holds no token of a sequence."""
    bs = case.k_pool.shape[2]
    held = torch.zeros(case.num_blocks, bs, dtype=torch.bool)
    for b, L in enumerate(case.lengths.tolist()):
        for t in range(L):
            held[case.block_tables[b, t // bs], t % bs] = True
    gap = ~held[:, None, :, None].expand_as(case.k_pool)
    case.k_pool[gap] = value
    case.v_pool[gap] = value
    return case


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_bounds(pa, dtype, d, bs):
    lens = [1, bs, bs + 1, 0, 5 * bs - 1, 7 * bs, 3]
    case = poison_past_lengths(custom_case(lens, 6, 3, d, bs, DT[dtype], seed=bs + d))
    tables = case.block_tables.tolist()
    start = torch.randn(case.num_blocks, 3, 2, d).to(DT[dtype])
    news = {"last token": None, "all": lens, "some": [1, 2, bs, 0, 2 * bs + 1, 0, 3]}
    for what, new in news.items():
        want = f64(start)
        rs.update_key_bounds(f64(case.k_pool), want, tables, lens, [min(L, 1) for L in lens] if new is None else new)
        got = start.cuda()
        qs = None if new is None else i32(np.concatenate([[0], np.cumsum(new)])).cuda()
        pa.pa_update_key_bounds(case.k_pool.cuda(), got, case.block_tables.cuda(), case.lengths.cuda(), query_start=qs,
                                max_query_len=1 if new is None else max(new))
        assert np.array_equal(f64(got), want), what
    assert pa.pa_read_error_flag() == 0


def test_bounds_of_shared_blocks(pa):
    """Sequences that share a prompt's full blocks: every one may bring them up to date."""
    k = torch.randn(7, 2, 8, 64).bfloat16()
    tables, lens = [[4, 1, 2], [4, 1, 5], [4, 1, 6]], [19, 24, 17]
    want = np.zeros((7, 2, 2, 64))
    rs.update_key_bounds(f64(k), want, tables, lens, lens)
    got = torch.zeros(7, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    pa.pa_update_key_bounds(k.cuda(), got, i32(tables).cuda(), i32(lens).cuda(),
                            query_start=i32([0, 19, 43, 60]).cuda(), max_query_len=24)
    assert np.array_equal(f64(got), want)
    assert pa.pa_read_error_flag() == 0


def test_bounds_special_values(pa):
    """NaN keys give NaN; infinities and zeros of both signs keep their order."""
    k = torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16)
    k[0, 0, 1, 3] = float("nan")
    k[0, 0, 5, 4] = float("inf")
    k[0, 0, 2, 5] = -float("inf")
    k[1] = torch.arange(8)[:, None] - 3.0
    kb = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    pa.pa_update_key_bounds(k.cuda(), kb, i32([[0], [1]]).cuda(), i32([8, 8]).cuda(), query_start=i32([0, 8, 16]).cuda(),
                            max_query_len=8)
    got = kb.cpu().float()
    assert got[0, 0, :, 3].isnan().all()
    assert got[0, 0, :, 4].tolist() == [0.0, float("inf")] and got[0, 0, :, 5].tolist() == [-float("inf"), 0.0]
    assert (got[1, 0, 0] == -3).all() and (got[1, 0, 1] == 4).all()


def test_bounds_bad_sequences(pa):
    k = torch.ones(4, 2, 8, 64, device="cuda")
    tables = i32([[0], [1], [4], [2], [3]]).cuda()
    lens = i32([4, 9, 8, -1, 8]).cuda()   # past its table, block past the pool, negative
    kb = torch.zeros(4, 2, 2, 64, device="cuda")
    pa.pa_update_key_bounds(k, kb, tables, lens)
    assert pa.pa_read_error_flag() == 5
    assert kb[0].eq(1).all() and kb[3].eq(1).all() and not kb[1:3].any()
    # more new tokens than the length, than the bound, and fewer than none
    for starts, maxq in (([0, 5, 5, 5, 5, 5], 8), ([0, 3, 3, 3, 3, 3], 2), ([3, 0, 0, 0, 0, 0], 8)):
        kb.zero_()
        pa.pa_update_key_bounds(k, kb, tables, i32([4, 0, 0, 0, 0]).cuda(), query_start=i32(starts).cuda(),
                                max_query_len=maxq)
        assert pa.pa_read_error_flag() == 5 and not kb.any()


# ---------------------------------------------------------------------------
# scores
# ---------------------------------------------------------------------------
def score_inputs(lens, hq, hkv, d, bs, dtype, seed=0):
    case = custom_case(lens, hq, hkv, d, bs, DT[dtype], seed=seed)
    g = torch.Generator().manual_seed(seed + 5)
    mid = torch.randn(case.num_blocks, hkv, d, generator=g)
    wide = torch.randn(case.num_blocks, hkv, d, generator=g).abs()
    return case, torch.stack([mid - wide, mid + wide], 2).to(DT[dtype])


def check_scores(pa, case, kb, bs, seqs=None, lens=None, width=None):
    q = case.q if seqs is None else torch.randn(len(seqs), *case.q.shape[1:]).to(case.q.dtype)
    lens = case.lengths.tolist() if lens is None else lens
    hkv, d = kb.shape[1], kb.shape[3]
    max_len = max(lens)
    S = -(-max_len // bs) + 3 if width is None else width
    want = np.full((len(lens), hkv, S), -7.0)
    size = rs.block_scores(f64(q), f64(kb), case.block_tables.tolist(), list(range(len(lens))) if seqs is None else seqs,
                           lens, bs, want)
    got = torch.full((len(lens), hkv, S), -7.0, device="cuda")
    pa.pa_block_scores(q.cuda(), kb.cuda(), case.block_tables.cuda(), i32(lens).cuda(), max_len, bs, got,
                       seq_ids=None if seqs is None else i32(seqs).cuda())
    err = np.abs(f64(got) - want)
    assert (err <= (2 * d + 2) * 2.0 ** -23 * size).all(), float(err.max())
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
def test_scores(pa, dtype, d, group):
    if group == 16 and dtype == "f32":
        pytest.skip("a group of 16 is bf16 only")
    bs = {1: 8, 2: 16, 4: 32, 8: 16, 16: 16}[group]
    lens = [1, 0, bs, 33 * bs - 1, 16 * bs, 17 * bs + 1, 100 * bs, 2]
    case, kb = score_inputs(lens, 3 * group, 3, d, bs, dtype, seed=group)
    check_scores(pa, case, kb, bs)
    assert pa.pa_read_error_flag() == 0


def test_scores_of_several_rows_a_sequence(pa):
    case, kb = score_inputs([40, 300], 8, 2, 128, 16, "bf16")
    check_scores(pa, case, kb, 16, seqs=[1, 1, 0, 1, 0], lens=[298, 299, 40, 300, 1])
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hkv,rows", [(1, 3), (2, 2), (5, 200), (8, 40)])
def test_scores_of_batches_and_head_counts(pa, dtype, hkv, rows):
    """Head counts that leave warps of a CTA without a head, and batches on both
    sides of each choice of tiles a warp."""
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, 700, (rows,), generator=g).tolist()
    case, kb = score_inputs(lens, 2 * hkv, hkv, 64, 8, dtype, seed=hkv)
    check_scores(pa, case, kb, 8)
    assert pa.pa_read_error_flag() == 0


def test_scores_of_a_long_row_among_short_ones(pa):
    case, kb = score_inputs([30000, 1, 700, 0, 12345], 4, 2, 64, 8, "bf16", seed=6)
    check_scores(pa, case, kb, 8)
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 4), (64, 16)])
def test_scores_of_many_long_rows(pa, dtype, d, group):
    """Several tiles a warp, through the ring of two."""
    if group == 16 and dtype == "f32":
        pytest.skip("a group of 16 is bf16 only")
    case, kb = score_inputs([30000, 17000], 2 * group, 2, d, 8, dtype, seed=7)
    seqs = [0, 1, 0, 0, 1, 0, 0, 1, 0, 0, 0, 1]
    lens = [30000, 17000, 29993, 1, 16391, 129, 0, 8192, 30000, 25000, 2049, 16999]
    check_scores(pa, case, kb, 8, seqs=seqs, lens=lens)
    assert pa.pa_read_error_flag() == 0


def test_scores_bad_rows_and_special_values(pa):
    case, kb = score_inputs([64, 64], 4, 2, 64, 16, "bf16")
    tables = case.block_tables.clone()
    tables[1, 2] = case.num_blocks
    kb = kb.cuda()
    seqs = i32([0, 2, -1, 1, 0, 0]).cuda()
    lens = i32([64, 64, 64, 64, 65, -1]).cuda()
    q = torch.ones(6, 4, 64, dtype=torch.bfloat16, device="cuda")
    got = torch.full((6, 2, 4), -7.0, device="cuda")
    pa.pa_block_scores(q, kb, tables.cuda(), lens, 64, 16, got, seq_ids=seqs)
    assert pa.pa_read_error_flag() == 5
    assert (got[[1, 2, 4, 5]] == -7).all() and (got[0] != -7).all()
    assert (got[3, :, [0, 1, 3]] != -7).all() and (got[3, :, 2] == -7).all()
    # a NaN query or bound makes its scores NaN and no others
    q[0, 3, 5] = float("nan")
    kb[tables[0, 1], 0, 0, 7] = float("nan")
    q[3] = -1
    pa.pa_block_scores(q, kb, tables.cuda(), i32([64, 0, 0, 16, 0, 0]).cuda(), 64, 16, got, seq_ids=i32([0] * 6).cuda())
    assert got[0, 1].isnan().all()
    assert not got[0, 0, [0, 2, 3]].isnan().any() and not got[3, :, 0].isnan().any()
    q[0, 3, 5], q[0, 0] = 1.0, -1.0    # a negative query reads the lower bound
    pa.pa_block_scores(q, kb, tables.cuda(), i32([64, 0, 0, 16, 0, 0]).cuda(), 64, 16, got, seq_ids=i32([0] * 6).cuda())
    assert got[0, 0].isnan().tolist() == [False, True, False, False]
    assert pa.pa_read_error_flag() == 0


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------
def check_select(pa, scores, lens, bs, K, first, last, max_len=None):
    want = rs.select_blocks(scores.numpy(), lens, bs, K, first, last)
    got = torch.full(tuple(want.shape), 99, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(scores.cuda(), i32(lens).cuda(), max(lens) if max_len is None else max_len, bs, got,
                        num_first=first, num_last=last)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["normal", "grid", "equal", "special", "ascending"])
@pytest.mark.parametrize("K,first,last", [(1, 0, 0), (1, 0, 1), (5, 1, 2), (64, 1, 2), (64, 64, 0), (200, 1, 1)])
@pytest.mark.parametrize("S", [200, 331, 2100])  # a warp, 512 and 1024 threads a row
def test_select(pa, kind, K, first, last, S):
    bs, R, hkv = 8, 9, 3
    g = torch.Generator().manual_seed(K)
    scores = torch.randn(R, hkv, S, generator=g) * 20
    if kind == "grid":
        scores = torch.round(scores / 8)
    elif kind == "equal":
        scores[:] = -3.5
    elif kind == "special":
        pick = torch.randint(0, 8, scores.shape, generator=g)
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45)):
            scores[pick == i] = x
    elif kind == "ascending":
        scores = torch.arange(S).float().expand(R, hkv, S).contiguous()
    blocks = [0, 1, 2, K, K + 1, 255, 257, S, 300]
    lens = [max(0, min(n, S) * bs - (i % bs if n else 0)) for i, n in enumerate(blocks)]
    check_select(pa, scores, lens, bs, K, first, last)
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("S", [1000, 4097, 20000, 70000])
def test_select_long_rows(pa, S):
    g = torch.Generator().manual_seed(S)
    scores = torch.randn(2, 2, S + 3, generator=g)
    scores[1] = torch.round(scores[1] * 4) / 4
    for K in (3, 256, 2047):
        check_select(pa, scores, [S * 16, S * 16 - 5], 16, K, 1, 2)
    assert pa.pa_read_error_flag() == 0


def test_arguments_of_the_wrong_kind(pa):
    """Refused by name before anything runs; numbers may be anything that counts."""
    scores, lens = torch.zeros(2, 1, 5, device="cuda"), i32([40, 33]).cuda()
    out = torch.full((2, 1, 4), 7, dtype=torch.int32, device="cuda")
    for bad, kind, what in (((scores.double(), lens, 40, 8, out), TypeError, "scores must be torch.float32"),
                            ((scores, lens.long(), 40, 8, out), TypeError, "context_lens must be torch.int32"),
                            ((scores, lens.cpu(), 40, 8, out), TypeError, "context_lens must be a CUDA tensor"),
                            ((scores, lens, 40, 8, out.transpose(0, 2).contiguous().transpose(0, 2)), ValueError,
                             "selected must be contiguous"),
                            ((scores, lens, 1 << 40, 8, out), OverflowError, "out of range"),
                            ((scores, lens, "40", 8, out), TypeError, "integer")):
        with pytest.raises(kind, match=what):
            pa.pa_select_blocks(*bad)
    with pytest.raises(TypeError):
        pa.pa_select_blocks(scores, lens, 40.5, 8, out)
    assert (out == 7).all()
    pa.pa_select_blocks(torch.nn.Parameter(scores), lens, np.int64(40), torch.tensor(8), out)
    assert out[:, 0].tolist() == [[0, 1, 3, 4]] * 2
    assert pa.pa_read_error_flag() == 0


def test_select_bad_lengths(pa):
    scores = torch.randn(3, 2, 10)
    got = torch.full((3, 2, 4), 99, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(scores.cuda(), i32([-1, 161, 160]).cuda(), 160, 16, got)
    assert pa.pa_read_error_flag() == 5
    assert (got[:2] == -1).all() and np.array_equal(got[2:].cpu().numpy(), rs.select_blocks(scores[2:].numpy(), [160],
                                                                                            16, 4, 1, 2))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def random_lists(case, hkv, K, seed=0, seqs=None, lens=None):
    """Distinct blocks of each row in random order, with gaps."""
    rng = np.random.default_rng(seed)
    bs = case.k_pool.shape[2]
    lens = case.lengths.tolist() if lens is None else lens
    out = np.full((len(lens), hkv, K), -1, np.int32)
    for r, L in enumerate(lens):
        n = -(-L // bs)
        for g in range(hkv):
            take = rng.permutation(n)[: K - (K > 3)]
            out[r, g, np.sort(rng.permutation(K)[: len(take)])] = take
    return out


def check_sparse(pa, case, lists, out_dtype=torch.float32, seqs=None, lens=None, q=None, what=""):
    q = case.q if q is None else q
    lens = case.lengths.tolist() if lens is None else lens
    clean = lambda t: np.nan_to_num(f64(t))  # poisoned places are masked: the definition never reads them
    want = rs.sparse_decode(f64(q), clean(case.k_pool), clean(case.v_pool), case.block_tables.tolist(),
                            list(range(len(lens))) if seqs is None else seqs, lens, lists.tolist(), case.scale)
    out = torch.full(tuple(q.shape), float("nan"), dtype=out_dtype, device="cuda")
    pa.pa_paged_attention_decode_sparse(q.cuda(), case.k_pool.cuda(), case.v_pool.cuda(), case.block_tables.cuda(),
                                        i32(lens).cuda(), torch.from_numpy(lists).cuda(), case.scale, out,
                                        seq_ids=None if seqs is None else i32(seqs).cuda())
    assert_matches_oracle(out, want, case.q.dtype == torch.bfloat16, what)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
def test_sparse_decode(pa, dtype, d, bs, group):
    if group == 16 and dtype == "f32":
        pytest.skip("a group of 16 is bf16 only")
    lens = [1, 0, bs - 1, bs + 1, 9 * bs - 3, 40 * bs, 61 * bs + 5]
    case = poison_past_lengths(custom_case(lens, 3 * group, 3, d, bs, DT[dtype], seed=group + bs))
    for K in (1, 7, 33):
        check_sparse(pa, case, random_lists(case, 3, K, seed=K), what=f"K {K}")
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sparse_decode_bf16_output(pa, dtype):
    case = custom_case([200, 77, 0, 500], 8, 2, 128, 16, DT[dtype], seed=2)
    check_sparse(pa, case, random_lists(case, 2, 20), torch.bfloat16)
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 3, 40, 400])
@pytest.mark.parametrize("K", [2, 65, 300])
def test_few_and_many_rows(pa, dtype, rows, K):
    """From one row, whose list is split over many CTAs, to more than the SMs hold."""
    n = 5
    case = custom_case([5000, 4093, 3000, 40, 1], 4, 1, 64, 16, DT[dtype], seed=rows)
    g = torch.Generator().manual_seed(3)
    seqs = [r % n for r in range(rows)]
    lens = [max(1, case.lengths[s].item() - r // n) for r, s in enumerate(seqs)]
    q = torch.randn(rows, 4, 64, generator=g).to(DT[dtype])
    check_sparse(pa, case, random_lists(case, 1, K, lens=lens), seqs=seqs, lens=lens, q=q)
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_block_is_dense_decode(pa, dtype):
    case = custom_case([1000, 333, 16, 2047], 8, 2, 128, 16, DT[dtype], seed=6)
    want = oracle.paged_decode(np_of(case.q), np_of(case.k_pool), np_of(case.v_pool), np_of(case.block_tables),
                               np_of(case.lengths), case.scale, 16)
    every = torch.arange(128, dtype=torch.int32).expand(4, 2, 128).clone()
    every[every >= -(-case.lengths[:, None, None] // 16)] = -1
    out = torch.empty(tuple(case.q.shape), device="cuda")
    pa.pa_paged_attention_decode_sparse(case.q.cuda(), case.k_pool.cuda(), case.v_pool.cuda(), case.block_tables.cuda(),
                                        case.lengths.cuda(), every.cuda(), case.scale, out)
    assert_matches_oracle(out, want, dtype == "bf16")
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lists(pa, dtype):
    """No entry, one entry twice, and the same blocks in another order."""
    case = custom_case([300, 300, 40], 4, 2, 128, 16, DT[dtype], seed=9)
    none = np.full((3, 2, 5), -1, np.int32)
    assert not check_sparse(pa, case, none).any()
    twice = none.copy()
    twice[:, :, 1:4] = [2, 0, 2]
    check_sparse(pa, case, twice)
    twice[0, 0, :] = 1      # one block five times is that block
    a = check_sparse(pa, case, twice)
    none[:, :, 2] = 1
    b = check_sparse(pa, case, none)
    assert (a[0, :2] - b[0, :2]).abs().max() <= 1e-5
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 40.0])
def test_scales(pa, dtype, scale):
    """Equal weights, a negative scale, and scores far beyond exp's range."""
    case = custom_case([300, 17], 8, 2, 64, 16, DT[dtype], seed=10)
    case.scale = float(np.float32(scale))
    if scale == 40.0:
        # whole-number vectors: the scores, up to thousands, are exact, and
        # distinct ones lie 40 apart, so a row is one token's value or a mean
        case.q = torch.randint(-2, 3, case.q.shape, generator=torch.Generator().manual_seed(1)).to(case.q.dtype)
        case.k_pool = torch.randint(-2, 3, case.k_pool.shape,
                                    generator=torch.Generator().manual_seed(2)).to(case.q.dtype)
    check_sparse(pa, case, random_lists(case, 2, 9))
    assert pa.pa_read_error_flag() == 0


def test_runs_alike_and_blocks_may_move(pa):
    """The same bits on every run, and under another placement of the blocks."""
    case = custom_case([900, 2000], 8, 2, 128, 16, torch.bfloat16, seed=12)
    lists = random_lists(case, 2, 50)
    a = check_sparse(pa, case, lists)
    assert torch.equal(a, check_sparse(pa, case, lists))
    perm = torch.randperm(case.num_blocks, generator=torch.Generator().manual_seed(5))
    case.k_pool[perm], case.v_pool[perm] = case.k_pool.clone(), case.v_pool.clone()
    case.block_tables = torch.where(case.block_tables >= 0, perm[case.block_tables.clamp(min=0).long()].int(), -1)
    assert torch.equal(a, check_sparse(pa, case, lists))
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sparse_bad_rows_and_entries(pa, dtype):
    case = custom_case([100, 64, 50], 4, 2, 64, 16, DT[dtype], seed=13)
    tables = case.block_tables.clone()
    tables[1, 2] = case.num_blocks   # outside the pool
    tables[1, 3] = -5
    lists = np.zeros((6, 2, 4), np.int32)
    lists[:] = [0, 1, -1, -1]
    lists[0] = [1, 7, 0, 1 << 30]    # past the row's 7 blocks
    lists[1] = [0, 2, 3, 1]
    seqs, lens = [0, 1, 3, -1, 2, 2], [100, 64, 10, 10, -1, 200]
    out = torch.full((6, 4, 64), float("nan"), device="cuda")
    q = torch.randn(6, 4, 64).to(DT[dtype])
    pa.pa_paged_attention_decode_sparse(q.cuda(), case.k_pool.cuda(), case.v_pool.cuda(), tables.cuda(), i32(lens).cuda(),
                                        torch.from_numpy(lists).cuda(), case.scale, out, seq_ids=i32(seqs).cuda())
    assert pa.pa_read_error_flag() == 5
    assert not out[2:].any()
    fine = np.full((2, 2, 4), -1, np.int32)
    fine[:] = [0, 1, -1, -1]
    want = rs.sparse_decode(f64(q[:2]), f64(case.k_pool), f64(case.v_pool), tables.tolist(), [0, 1], [100, 64],
                            fine.tolist(), case.scale)
    assert_matches_oracle(out[:2], want, dtype == "bf16")


def test_pool_beyond_32_bits(pa):
    """Blocks whose element offsets pass 2^31 and 2^32, through every call of the step."""
    NB, hkv, bs, d = 270_000, 8, 16, 128          # 4.4e9 elements a pool
    kp = torch.zeros(NB, hkv, bs, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros(NB, hkv, bs, d, dtype=torch.bfloat16, device="cuda")
    small = custom_case([40], 8, 8, d, bs, torch.bfloat16, seed=4, extra_blocks=0)
    far = i32([[NB - 1, NB // 2 + 7, 3]])
    for j in range(3):
        kp[far[0, j]] = small.k_pool[small.block_tables[0, j]].cuda()
        vp[far[0, j]] = small.v_pool[small.block_tables[0, j]].cuda()
    kb = torch.zeros(NB, hkv, 2, d, dtype=torch.bfloat16, device="cuda")
    lens = i32([40]).cuda()
    pa.pa_update_key_bounds(kp, kb, far.cuda(), lens, query_start=i32([0, 40]).cuda(), max_query_len=40)
    skb = torch.zeros(3, hkv, 2, d, dtype=torch.bfloat16, device="cuda")
    pa.pa_update_key_bounds(small.k_pool.cuda(), skb, small.block_tables.cuda(), lens,
                            query_start=i32([0, 40]).cuda(), max_query_len=40)
    for j in range(3):
        assert torch.equal(kb[far[0, j]], skb[small.block_tables[0, j]])
    res = []
    for k, v, b, t in ((kp, vp, kb, far.cuda()), (small.k_pool.cuda(), small.v_pool.cuda(), skb,
                                                  small.block_tables.cuda())):
        scores = torch.zeros(1, hkv, 4, device="cuda")
        sel = torch.zeros(1, hkv, 2, dtype=torch.int32, device="cuda")
        out = torch.zeros(1, 8, d, device="cuda")
        pa.pa_block_scores(small.q.cuda(), b, t, lens, 40, bs, scores)
        pa.pa_select_blocks(scores, lens, 40, bs, sel, num_first=0, num_last=1)
        pa.pa_paged_attention_decode_sparse(small.q.cuda(), k, v, t, lens, sel, small.scale, out)
        res.append((scores, sel, out))
    assert all(torch.equal(x, y) for x, y in zip(*res)) and res[0][2].any()
    # the cache write at the far end
    cs = torch.cat([torch.ones(64, 64), torch.zeros(64, 64)], 1).cuda()
    key = torch.randn(1, hkv, d, device="cuda").bfloat16()
    qo = torch.empty_like(key)
    pa.pa_rope_and_cache(key, key, key, qo, kp, vp, torch.tensor([NB * bs - 1], device="cuda"), i32([5]).cuda(), cs)
    assert torch.equal(kp[NB - 1, :, bs - 1], key[0]) and torch.equal(vp[NB - 1, :, bs - 1], key[0])
    assert torch.equal(qo, key) and pa.pa_read_error_flag() == 0


# ---------------------------------------------------------------------------
# the calls together
# ---------------------------------------------------------------------------
class Model:
    """One attention layer's decode state on the GPU and its fp64 twin."""

    def __init__(self, pa, lens, hq, hkv, d, bs, dtype, K, seed=0, steps=4):
        self.pa, self.hq, self.hkv, self.d, self.bs, self.dtype, self.K = pa, hq, hkv, d, bs, dtype, K
        self.scale = float(np.float32(1 / math.sqrt(d)))
        self.max_len = max(lens) + steps
        case = custom_case([L + steps for L in lens], hq, hkv, d, bs, DT[dtype], seed=seed)
        self.tables, self.k_pool, self.v_pool = case.block_tables.cuda(), case.k_pool.cuda(), case.v_pool.cuda()
        self.lens = i32(lens).cuda()
        g = torch.Generator().manual_seed(seed)
        freq = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d)
        a = torch.arange(self.max_len, dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()
        self.qw, self.kw = ((1 + 0.1 * torch.randn(d, generator=g)).to(DT[dtype]).cuda() for _ in range(2))
        B = len(lens)
        self.kb = torch.zeros(case.num_blocks, hkv, 2, d, dtype=DT[dtype], device="cuda")
        self.query_out = torch.zeros(B, hq, d, dtype=DT[dtype], device="cuda")
        self.scores = torch.zeros(B, hkv, -(-self.max_len // bs), device="cuda")
        self.selected = torch.zeros(B, hkv, K, dtype=torch.int32, device="cuda")
        self.out = torch.zeros(B, hq, d, device="cuda")
        self.slots = torch.zeros(B, dtype=torch.int64, device="cuda")
        self.qkv = torch.zeros(B, hq + 2 * hkv, d, dtype=DT[dtype], device="cuda")
        starts = i32(np.concatenate([[0], np.cumsum(lens)])).cuda()
        pa.pa_update_key_bounds(self.k_pool, self.kb, self.tables, self.lens, query_start=starts, max_query_len=max(lens))

    def step(self, stream=None):
        hq, hkv = self.hq, self.hkv
        self.pa.sparse_decode_step(self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:], self.k_pool,
                                   self.v_pool, self.kb, self.tables, self.lens, self.max_len, self.cos_sin, self.scale,
                                   self.query_out, self.scores, self.selected, self.out, q_weight=self.qw,
                                   k_weight=self.kw, slots=self.slots, stream=stream)

    def check(self):
        """Each stage against its definition on the GPU's own inputs to it."""
        lens, tables, B = self.lens.tolist(), self.tables.tolist(), self.lens.numel()
        bounds = f64(self.kb)
        rs.update_key_bounds(f64(self.k_pool), bounds, tables, lens, lens)
        assert np.array_equal(bounds, f64(self.kb))  # the running update is the whole recomputation
        want = f64(self.scores)
        size = rs.block_scores(f64(self.query_out), bounds, tables, range(B), lens, self.bs, want)
        assert (np.abs(f64(self.scores) - want) <= (2 * self.d + 2) * 2.0 ** -23 * size).all()
        want = rs.select_blocks(self.scores.cpu().numpy(), lens, self.bs, self.K, 1, 2)
        assert np.array_equal(self.selected.cpu().numpy(), want)
        want = rs.sparse_decode(f64(self.query_out), f64(self.k_pool), f64(self.v_pool), tables, range(B), lens,
                                want.tolist(), self.scale)
        assert_matches_oracle(self.out, want, self.dtype == "bf16")
        assert self.pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", [("bf16", 8, 2, 128, 16), ("f32", 4, 4, 64, 8), ("bf16", 16, 1, 64, 32)])
@pytest.mark.parametrize("K", [6, 1000])
def test_sparse_decode_steps(pa, dtype, hq, hkv, d, bs, K):
    """Several steps of a batch, the first eager, the rest from one graph; with a
    budget above every context it is the dense step."""
    steps = 4
    m = Model(pa, [301, 15, 128, 1000], hq, hkv, d, bs, dtype, K, steps=steps)
    g = torch.Generator().manual_seed(7)
    graph = None
    for i in range(steps):
        m.qkv.copy_(torch.randn(m.qkv.shape, generator=g))
        m.lens += 1
        before = m.k_pool.clone()
        if i == 0:
            m.step()
        elif graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                m.step()
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        m.check()
        # the step wrote one slot of each sequence and nothing else
        changed = (m.k_pool != before).any(dim=(1, 3)).nonzero()
        assert sorted((changed[:, 0] * bs + changed[:, 1]).tolist()) == sorted(m.slots.tolist())
        if K == 1000:
            dense = torch.zeros_like(m.out)
            pa.pa_paged_attention_decode(m.query_out, m.k_pool, m.v_pool, m.tables, m.lens, m.max_len, m.scale, dense)
            bar = 2e-5 if dtype == "f32" else 4e-3  # each within its bar of the same fp64 value
            assert (m.out - dense).abs().max().item() <= bar


def test_two_streams_at_once(pa):
    """Two layers' steps on two streams, interleaved, end as each does alone."""
    models = [Model(pa, [700, 90, 1500], 8, 2, 128, 16, "bf16", 12, seed=s) for s in (1, 2)]
    g = torch.Generator().manual_seed(3)
    for m in models:
        m.qkv.copy_(torch.randn(m.qkv.shape, generator=g))
        m.lens += 1
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for m, s in zip(models, streams):
            m.step(stream=s)
    torch.cuda.synchronize()
    for m in models:
        m.check()
