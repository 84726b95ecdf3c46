"""Plain numpy fp64 definitions of the rotary cache write and of block-sparse
decode attention: explicit loops over tokens, heads and blocks, sharing no code
with the product package.  Arrays of values are float64 (already widened by the
caller); tables, lengths and lists are integer arrays.
"""
from __future__ import annotations

import numpy as np


def norm_rotate(x, weight, eps, angles, interleaved):
    """One head row x [D] in fp64; weight [D] or None; angles: list of (c, s),
    one a pair of the first 2 * len(angles) elements.  Returns the row and, per
    element, the sum of magnitudes its last step adds (for error bounds)."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).sum() / x.size + eps) * weight
    out, size = x.copy(), np.abs(x)
    half = len(angles)
    for p, (c, s) in enumerate(angles):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        out[a] = x[a] * c - x[b] * s
        out[b] = x[b] * c + x[a] * s
        size[a] = abs(x[a] * c) + abs(x[b] * s)
        size[b] = abs(x[b] * c) + abs(x[a] * s)
    return out, size


def pair_angles(cos_sin, positions, token, pair_axes):
    """(c, s) of every pair of one token; positions [axes, tokens]."""
    half = cos_sin.shape[1] // 2
    out = []
    for p in range(half):
        axis = 0 if pair_axes is None else int(pair_axes[p])
        row = cos_sin[int(positions[axis, token])]
        out.append((float(row[p]), float(row[half + p])))
    return out


def rope_and_cache(query, key, value, slots, positions, cos_sin, pair_axes, interleaved, q_weight, k_weight, eps,
                   query_out, k_pool, v_pool):
    """Writes into query_out [T, Hq, D] and the pools [NB, Hkv, bs, D] in place;
    returns arrays of the same shapes with each written element's size (0 where
    nothing is written).  Tokens with a negative slot write nothing."""
    q_size, k_size = np.zeros_like(query_out), np.zeros_like(k_pool)
    bs = k_pool.shape[2]
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        angles = pair_angles(cos_sin, positions, t, pair_axes)
        blk, off = int(slot) // bs, int(slot) % bs
        for h in range(query.shape[1]):
            query_out[t, h], q_size[t, h] = norm_rotate(query[t, h], q_weight, eps, angles, interleaved)
        for h in range(key.shape[1]):
            k_pool[blk, h, off], k_size[blk, h, off] = norm_rotate(key[t, h], k_weight, eps, angles, interleaved)
            v_pool[blk, h, off] = value[t, h]
    return q_size, k_size


def update_key_bounds(k_pool, key_bounds, tables, lens, new):
    """Recomputes in place the bounds of the blocks that hold each sequence's
    last new[b] tokens."""
    bs = k_pool.shape[2]
    for b, L in enumerate(lens):
        for j in sorted({t // bs for t in range(L - new[b], L)}):
            blk = tables[b][j]
            held = k_pool[blk, :, : min(bs, L - j * bs)]
            key_bounds[blk, :, 0] = held.min(axis=1)
            key_bounds[blk, :, 1] = held.max(axis=1)


def block_scores(q, key_bounds, tables, seqs, lens, block_size, scores):
    """Fills scores [R, Hkv, S] for each row's blocks; returns the largest sum
    of |terms| of each (for error bounds)."""
    hkv = key_bounds.shape[1]
    group = q.shape[1] // hkv
    size = np.zeros_like(scores)
    for r, L in enumerate(lens):
        for j in range(-(-L // block_size)):
            lo, hi = key_bounds[tables[seqs[r]][j], :, 0], key_bounds[tables[seqs[r]][j], :, 1]
            for g in range(hkv):
                terms = np.maximum(q[r, g * group:(g + 1) * group] * lo[g], q[r, g * group:(g + 1) * group] * hi[g])
                scores[r, g, j] = terms.sum(axis=1).max()
                size[r, g, j] = np.abs(terms).sum(axis=1).max()
    return size


def select_blocks(scores, lens, block_size, max_selected, num_first, num_last):
    """int32 [R, Hkv, max_selected], one row at a time by plain sorting."""
    out = np.full(scores.shape[:2] + (max_selected,), -1, np.int32)
    for r, L in enumerate(lens):
        n = -(-L // block_size)
        always = [j for j in range(n) if j < num_first or j >= n - num_last]
        for g in range(scores.shape[1]):
            row = scores[r, g]
            rest = [j for j in range(n) if j not in set(always)]
            rest.sort(key=lambda j: (0 if row[j] != row[j] else 1, -row[j] if row[j] == row[j] else 0.0, j))
            kept = sorted((always + rest)[:max_selected] if len(always) <= max_selected else [])
            out[r, g, : len(kept)] = kept
    return out


def sparse_decode(q, k_pool, v_pool, tables, seqs, lens, selected, scale):
    """fp64 [R, Hq, D]: softmax attention over the tokens of the listed blocks
    (a block listed twice counts twice, a negative entry names none)."""
    hkv, bs = k_pool.shape[1], k_pool.shape[2]
    group = q.shape[1] // hkv
    out = np.zeros(q.shape, np.float64)
    for r, L in enumerate(lens):
        for g in range(hkv):
            ks, vs = [], []
            for j in selected[r][g]:
                if j < 0:
                    continue
                blk = tables[seqs[r]][j]
                held = min(bs, L - j * bs)
                ks.append(k_pool[blk, g, :held])
                vs.append(v_pool[blk, g, :held])
            if not ks:
                continue
            ks, vs = np.concatenate(ks), np.concatenate(vs)
            for h in range(g * group, (g + 1) * group):
                s = scale * (ks @ q[r, h])
                w = np.exp(s - s.max())
                out[r, h] = (w / w.sum()) @ vs
    return out
