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
