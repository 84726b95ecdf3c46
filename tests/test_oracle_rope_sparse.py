"""Pins of the fp64 definitions of the rotary cache write and block-sparse
decode: closed forms, invariants and the dense oracle (no GPU)."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle
from oracle import rope_sparse as rs


def table(last, rotary, base=10000.0):
    freq = base ** (-np.arange(rotary // 2) * 2.0 / rotary)
    a = np.arange(last)[:, None] * freq
    return np.concatenate([np.cos(a), np.sin(a)], axis=1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_closed_forms(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal(64)
    cs = table(50, 32)
    # position 0 leaves a row as it is; so does every element past rotary_dim
    out, _ = rs.norm_rotate(x, None, 0.0, rs.pair_angles(cs, np.zeros((1, 1), int), 0, None), interleaved)
    assert np.array_equal(out, x)
    pos = np.array([[7, 12, 40, 45]])
    rows = [rs.norm_rotate(x, None, 0.0, rs.pair_angles(cs, pos, t, None), interleaved)[0] for t in range(4)]
    assert all(np.array_equal(r[32:], x[32:]) for r in rows)
    # a rotation keeps lengths, and dot products depend on the distance alone
    assert all(abs(np.linalg.norm(r) - np.linalg.norm(x)) < 1e-12 for r in rows)
    y = rng.standard_normal(64)
    other = [rs.norm_rotate(y, None, 0.0, rs.pair_angles(cs, pos, t, None), interleaved)[0] for t in range(4)]
    assert abs(rows[0] @ other[1] - rows[2] @ other[3]) < 1e-12
    # a quarter turn of one pair
    quarter, _ = rs.norm_rotate([3.0, 5.0, 1.0, 2.0], None, 0.0, [(0.0, 1.0), (1.0, 0.0)], interleaved)
    assert quarter.tolist() == ([-5.0, 3.0, 1.0, 2.0] if interleaved else [-1.0, 5.0, 3.0, 2.0])


def test_norm_closed_forms():
    x = np.array([3.0, -4.0, 0.0, 0.0])
    out, _ = rs.norm_rotate(x, np.ones(4), 0.0, [], False)
    assert np.allclose(out, x / math.sqrt(25 / 4), rtol=0, atol=1e-15)
    scaled, _ = rs.norm_rotate(100 * x, np.ones(4), 0.0, [], False)
    assert np.allclose(scaled, out, rtol=0, atol=1e-15)
    zero, _ = rs.norm_rotate(np.zeros(4), np.ones(4), 1e-6, [], False)
    assert np.array_equal(zero, np.zeros(4))


def test_pairs_turn_by_their_own_axis():
    cs = table(30, 16)
    pos = np.array([[3], [11], [20]])
    axes = np.array([0, 1, 2, 0, 1, 2, 0, 1])
    got = rs.pair_angles(cs, pos, 0, axes)
    for p, a in enumerate(axes):
        assert got[p] == (cs[pos[a, 0], p], cs[pos[a, 0], 8 + p])
    # equal positions on every axis are the single-axis rotation
    assert rs.pair_angles(cs, np.array([[9], [9], [9]]), 0, axes) == rs.pair_angles(cs, np.array([[9]]), 0, None)


def _case(seed=0, lens=(37, 5, 64), hq=4, hkv=2, d=8, bs=8):
    rng = np.random.default_rng(seed)
    need = [-(-L // bs) for L in lens]
    ids = rng.permutation(sum(need) + 3)
    tables = np.full((len(lens), max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at: at + n]
        at += n
    pool = lambda: rng.standard_normal((sum(need) + 3, hkv, bs, d))
    return rng, list(lens), tables, pool(), pool(), rng.standard_normal((len(lens), hq, d))


def test_scores_bound_every_dot_product_and_are_reached():
    rng, lens, tables, k, v, q = _case()
    bounds = np.zeros((k.shape[0], 2, 2, 8))
    rs.update_key_bounds(k, bounds, tables, lens, lens)
    scores = np.full((3, 2, 9), 7.0)
    rs.block_scores(q, bounds, tables, [0, 1, 2], lens, 8, scores)
    for b, L in enumerate(lens):
        for j in range(9):
            if j >= -(-L // 8):
                assert (scores[b, :, j] == 7.0).all()  # past the row's blocks: left as it was
                continue
            held = k[tables[b, j], :, : min(8, L - 8 * j)]
            for g in range(2):
                assert scores[b, g, j] >= (held[g] @ q[b, 2 * g: 2 * g + 2].T).max() - 1e-12
    # one token a block: the bound is the dot product itself
    one = k[:, :, :1]
    bounds = np.concatenate([one, one], axis=2)
    rs.block_scores(q, bounds, tables, [0, 1, 2], lens, 8, scores)
    assert abs(scores[0, 1, 2] - (one[tables[0, 2], 1, 0] @ q[0, 2:4].T).max()) < 1e-12


def test_selection_by_hand():
    row = np.array([[[1.0, 9.0, 9.0, 2.0, np.nan, 9.0, -np.inf, 0.5]]])
    pick = lambda n, K, first, last: rs.select_blocks(row, [n * 8], 8, K, first, last)[0, 0].tolist()
    assert pick(8, 3, 0, 0) == [1, 2, 4]        # NaN first, then the lower of the equal ones
    assert pick(8, 4, 1, 1) == [0, 1, 4, 7]
    assert pick(8, 4, 0, 4) == [4, 5, 6, 7]
    assert pick(3, 5, 1, 2) == [0, 1, 2, -1, -1]
    assert pick(0, 2, 1, 1) == [-1, -1]


def test_attending_to_every_block_is_dense_attention():
    rng, lens, tables, k, v, q = _case(3)
    k, v, q = (x.astype(np.float32) for x in (k, v, q))
    every = np.full((3, 2, 10), -1)
    for b, L in enumerate(lens):
        n = -(-L // 8)
        for g in range(2):
            every[b, g, rng.permutation(10)[:n]] = rng.permutation(n)  # any order, gaps anywhere
    want = oracle.paged_decode(q, k, v, tables, np.array(lens), 0.3, 8)
    got = rs.sparse_decode(q.astype(np.float64), k.astype(np.float64), v.astype(np.float64), tables, [0, 1, 2], lens,
                           every, float(np.float32(0.3)))
    assert np.abs(got - want).max() < 1e-12
    nothing = rs.sparse_decode(q, k, v, tables, [0, 1, 2], lens, np.full((3, 2, 4), -1), 0.3)
    assert not nothing.any()
