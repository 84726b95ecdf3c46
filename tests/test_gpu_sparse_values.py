"""GPU tests of what block-sparse decode attention does with single values: how
exactly a weight reaches the output, and where NaN and infinities of attended
tokens go."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import rope_sparse as rs

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


def attend(pa, q, kp, vp, tables, lens, lists, scale, out_dtype=torch.float32):
    out = torch.full(tuple(q.shape), 7.0, dtype=out_dtype, device="cuda")
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    pa.pa_paged_attention_decode_sparse(q.cuda(), kp.cuda(), vp.cuda(), i32(tables), i32(lens), i32(lists), scale, out)
    return out


@pytest.mark.parametrize("dtype,group", [("f32", 1), ("f32", 8), ("bf16", 1), ("bf16", 8), ("bf16", 16)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("rows,K", [(3, 4), (3, 128), (300, 4)])  # one CTA a list, several, four warps a CTA
def test_weights_reach_the_output_in_32_bits(pa, dtype, group, d, bs, rows, K):
    """Rows that attend to 16 tokens whose values are distinct unit vectors, so
    that an output element is one softmax weight and no sum of values hides its
    error; whole-number vectors and a scale of 2^-7, so that scores are exact.

    In units of 2^-24 of the element, with |score| log2(e) <= 1 (asserted): a
    weight's exponent x - m is off by the rounding of log2(e) (of at most 2),
    those of x and m (1 each) and that of the difference (2), together ln 2 * 6
    = 4.2; 2^x is off by 2^-22 = 4; the value product adds it in up to three
    parts, 4, and may lose the last part's end, 1: 13.2.  Where the 16 tokens are
    two warps' their parts are joined by another power of the same kind, ln 2 * 2
    + 4, and a product, 1: 6.4.  The sum of the weights has the weights' own
    8.2, those 6.4, and at most 8 additions, 8.  The division rounds once, 1.
    13.2 + 6.4 + 8.2 + 6.4 + 8 + 1 < 44."""
    g = torch.Generator().manual_seed(d + bs + group)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g).to(DT[dtype])
    per_row = max(1, 16 // bs)  # blocks of a row
    nb = rows * per_row
    q, kp = whole(rows, group, d), whole(nb, 1, bs, d)
    vp = torch.zeros(nb, 1, bs, d, dtype=DT[dtype])
    tables = torch.randperm(nb, generator=g).reshape(rows, per_row)
    for r in range(rows):
        for t in range(16):
            vp[tables[r, t // bs], 0, t % bs, 4 * t + 1] = 1
    lists = np.full((rows, 1, K), -1, np.int32)
    lists[:, 0, K // 2: K // 2 + per_row] = np.arange(per_row)  # both halves of one tile
    lens, scale = [16] * rows, 2.0 ** -7
    out = f64(attend(pa, q, kp, vp, tables, lens, lists, scale))
    for r in range(0, rows, 1 if rows < 10 else 37):
        k = np.concatenate([f64(kp[b, 0]) for b in tables[r]])[:16]
        assert np.abs(f64(q[r]) @ k.T).max() * scale * math.log2(math.e) <= 1
        want = rs.sparse_decode(f64(q[r:r + 1]), f64(kp), f64(vp), [tables[r].tolist()], [0], [16],
                                lists[r:r + 1].tolist(), scale)[0]
        assert ((want > 0).sum(axis=1) == 16).all()
        err = np.abs(out[r] - want)
        assert (err <= 44 * 2.0 ** -24 * want).all(), float((err / np.where(want > 0, want, 1)).max() * 2.0 ** 24)
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype,group", [("f32", 1), ("bf16", 1), ("bf16", 8), ("bf16", 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_long_lists_have_no_drift(pa, dtype, group, d):
    """160 rows that attend to 16,384 tokens each with positive values, one CTA a
    list: about 170 tiles a warp.  Sums rounded to nearest scatter about the
    definition (over the 10,000 and more elements here their mean is off by less
    than 2^-24 of the value), sums that are cut off drift to one side, by about
    0.36 * 2^-23 of what is held each time.  A tile's own products may be cut off
    (three sums of at most 17 addends, the largest an eighth of the sum or so:
    3 * 17 / 8 * 2^-23 / 2 = 6.4 * 2^-24); a running sum that is cut off twice a
    tile would be 0.36 * 170 * 2^-23 = 122 * 2^-24 below."""
    g = torch.Generator().manual_seed(d + group)
    bs, n, rows = 16, 1024, 160
    q = torch.randn(rows, group, d, generator=g).to(DT[dtype])
    kp = torch.randn(n, 1, bs, d, generator=g).to(DT[dtype])
    vp = (1 + torch.rand(n, 1, bs, d, generator=g)).to(DT[dtype])
    table = torch.randperm(n, generator=g).to(torch.int32)
    out = torch.zeros(rows, group, d, device="cuda")
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    pa.pa_paged_attention_decode_sparse(q.cuda(), kp.cuda(), vp.cuda(), table[None].cuda(), i32([n * bs] * rows),
                                        torch.arange(n, dtype=torch.int32).expand(rows, 1, n).contiguous().cuda(), 0.125, out,
                                        seq_ids=i32([0] * rows))
    k, v = (p[table.long(), 0].reshape(n * bs, d).double().cuda() for p in (kp, vp))
    want = torch.softmax(q.double().cuda() @ k.T * 0.125, dim=-1) @ v
    off = (out.double() / want - 1).mean().item() * 2.0 ** 24
    assert abs(off) <= 16, off
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [4, 100])  # one CTA a list, several
def test_nan_and_infinities_of_attended_tokens(pa, dtype, K):
    """They go where the formula sends them, and nowhere else."""
    g = torch.Generator().manual_seed(K)
    rows, hkv, group, d, bs, L = 7, 2, 4, 64, 16, 60
    draw = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])
    tables = torch.randperm(rows * 4 + 2, generator=g)[: rows * 4].reshape(rows, 4)
    q, kp, vp = draw(rows, hkv * group, d), draw(rows * 4 + 2, hkv, bs, d), draw(rows * 4 + 2, hkv, bs, d)
    lists = np.full((rows, hkv, K), -1, np.int32)
    lists[:, :, :3] = [3, 0, 2]                        # block 1 is not attended to
    nan, inf = float("nan"), float("inf")
    heads = lambda h: slice(h * group, (h + 1) * group)
    scale = 0.125
    clean = rs.sparse_decode(f64(q), f64(kp), f64(vp), tables.tolist(), range(rows), [L] * rows, lists.tolist(), scale)
    kp[tables[0, 2], 0, 5, 7] = nan                    # row 0, kv head 0: every score's head, all channels
    vp[tables[1, 0], 1, 3, 9] = nan                    # row 1, kv head 1: one channel
    vp[tables[2, 3], 0, 11, 20] = inf                  # row 2: the last attended token's value
    kp[tables[3, 2], 1, 0, 0] = -inf                   # row 3: a score of -inf, a weight of 0
    q[3, heads(1), 0] = 1.0
    kp[tables[4, 0], 0, 2, 0], q[4, heads(0), 0] = inf, 0.5   # row 4: a score of +inf
    q[5, 2, 1] = nan                                   # row 5: one query head
    for b, h in ((tables[6, 1], 0), (tables[6, 1], 1)):       # row 6: a block that is not listed, and past the length
        kp[b, h], vp[b, h] = nan, inf
    kp[tables[6, 3], :, 12:], vp[tables[6, 3], :, 12:] = nan, inf
    out = f64(attend(pa, q, kp, vp, tables, [L] * rows, lists, scale))
    with np.errstate(invalid="ignore"):
        want = rs.sparse_decode(f64(q), f64(kp), f64(vp), tables.tolist(), range(rows), [L] * rows, lists.tolist(), scale)
    assert np.isnan(want[0, :4]).all() and np.isfinite(want[0, 4:]).all()
    assert np.isnan(want[1, 4:, 9]).all() and np.isnan(want).sum() == 4 * d + 4 + 4 * d + d
    assert (want[2, :4, 20] == inf).all() and np.isfinite(want[3]).all() and np.isnan(want[4, :4]).all()
    if dtype == "bf16":
        # an infinite V meets the weight's three parts: inf where all are positive, else inf - inf or 0 * inf
        assert not np.isfinite(out[2, :4, 20]).any() and not (out[2, :4, 20] == -inf).any()
        out[2, :4, 20] = want[2, :4, 20]
    finite = np.isfinite(want)
    assert np.array_equal(np.isnan(out), np.isnan(want)) and np.array_equal(out[np.isinf(want)], want[np.isinf(want)])
    bar = 1e-5 if dtype == "f32" else 2e-3
    assert np.abs(out[finite] - want[finite]).max() <= bar and np.array_equal(want[6], clean[6])
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [4, 100])
def test_all_scores_minus_infinity_give_zeros(pa, dtype, K):
    """No weight is left to share out: such a row is as one that attends to
    nothing, whichever other rows and heads are finite."""
    g = torch.Generator().manual_seed(3)
    draw = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])
    q, kp, vp = draw(3, 4, 64), draw(9, 2, 8, 64), draw(9, 2, 8, 64)
    q[:, :, 0] = 1.0
    tables = torch.arange(9).reshape(3, 3)
    kp[tables[1], 1, :, 0] = -float("inf")
    lists = np.full((3, 2, K), -1, np.int32)
    lists[:, :, 1:4] = [0, 1, 2]
    out = f64(attend(pa, q, kp, vp, tables, [24, 20, 3], np.where(lists * 8 < np.array([24, 20, 3])[:, None, None], lists, -1), 0.125))
    assert not out[1, 2:].any()
    out[1, 2:] = 1.0
    assert np.isfinite(out).all() and (out != 0).all()
    assert pa.pa_read_error_flag() == 0
