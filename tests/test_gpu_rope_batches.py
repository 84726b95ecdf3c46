"""GPU parity of the rotary cache write where one warp takes several batches of
a token's rows one after another: queries, then keys, then values, with other
weights from the keys on and a last batch of a kind that is in part empty.

Tolerances as in test_gpu_rope.py: 16 steps of 2^-24 of the magnitudes an
element's last step adds, and one rounding at the store.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import rope_sparse as rs

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def batches_of_a_warp(tokens, hq, hkv, d, dtype, sms):
    """The launch's plan: batches of rows that one warp takes."""
    per_step, most = 32 // (d // 8), 4 if dtype == "bf16" else 2
    up = lambda a, b: -(-a // b)
    steps = up(hq, per_step) + 2 * up(hkv, per_step)
    total = steps * tokens
    per_warp = total // (sms * 64)
    if per_warp < 4 and total >= sms * 32:
        per_warp = 4
    if per_warp < 16 and tokens * up(steps, 16) >= sms * 28:
        per_warp = 16
    per_warp = max(1, min(per_warp, steps))
    batch = min(per_warp, most)
    q, kv = up(hq, batch * per_step), up(hkv, batch * per_step)
    slices = up((q + 2 * kv) * batch, per_warp)
    return up(q + 2 * kv, slices)


@pytest.mark.parametrize("hq,hkv,d,tokens", [
    (32, 32, 128, 4700),   # four batches a warp, each of one kind
    (18, 9, 128, 2300),    # q and k in one warp, last batches in part empty
    (78, 10, 64, 2301),    # a warp with the last of q, k and v
    (64, 8, 128, 9500),    # a whole token a warp
])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rotary,interleaved,axes,norm", [
    ("whole", False, 1, (True, True)), ("whole", True, 3, (True, False)), ("part", False, 3, (False, True)),
    ("part", True, 1, (True, True)), ("whole", True, 1, (False, False))])
def test_several_batches_a_warp(hq, hkv, d, tokens, dtype, rotary, interleaved, axes, norm):
    import paged_kv_cache_355_b200 as pa

    each = batches_of_a_warp(tokens, hq, hkv, d, dtype,
                             torch.cuda.get_device_properties(0).multi_processor_count)
    assert each >= 4
    pa.pa_read_error_flag()
    g = torch.Generator(device="cuda").manual_seed(tokens + axes)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[dtype])
    R, bs, last = d if rotary == "whole" else d // 2 - 16, 16, 3000
    nb = tokens // bs + 5
    qkv, query_out = rnd(tokens, hq + 2 * hkv, d), rnd(tokens, hq, d)
    kp, vp = rnd(nb, hkv, bs, d), rnd(nb, hkv, bs, d)
    before = query_out.clone(), kp.clone(), vp.clone()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:tokens]
    slots[::11] = -1
    positions = torch.randint(0, last, (axes, tokens), generator=g, device="cuda", dtype=torch.int32)
    pair_axes = torch.randint(0, axes, (R // 2,), generator=g, device="cuda", dtype=torch.int32) if axes > 1 else None
    freq = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) * 2 / R)
    angle = torch.arange(last, dtype=torch.float64)[:, None] * freq
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(DT[dtype]) if on else None for on in norm]
    pa.pa_rope_and_cache(q, k, v, query_out, kp, vp, slots, positions, cos_sin.cuda(), pair_axes=pair_axes,
                         interleaved=interleaved, q_weight=w[0], k_weight=w[1])
    assert pa.pa_read_error_flag() == 0
    # values bit for bit, and what no token writes left as it was
    kept = slots >= 0
    flat = lambda p: p.transpose(1, 2).reshape(nb * bs, hkv, d)
    want_v = flat(before[2]).clone()
    want_v[slots[kept]] = v[kept]
    assert torch.equal(flat(vp), want_v)
    unwritten = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    unwritten[slots[kept]] = False
    assert torch.equal(flat(kp)[unwritten], flat(before[1])[unwritten])
    assert torch.equal(query_out[~kept], before[0][~kept])
    # queries and keys of some tokens, all heads, by their definition
    some = [t for t in list(range(1, 4)) + list(range(5, tokens, 811)) + [tokens - 2, tokens - 1] if slots[t] >= 0]
    at = torch.tensor(some, device="cuda")
    weights = [None if x is None else f64(x) for x in w]
    table, axis_of = f64(cos_sin), None if pair_axes is None else pair_axes.cpu().numpy()
    pos = positions.cpu().numpy()
    for got, src, weight in ((query_out[at], q[at], weights[0]), (flat(kp)[slots[at]], k[at], weights[1])):
        got, src = f64(got), f64(src)
        for i, t in enumerate(some):
            angles = rs.pair_angles(table, pos, t, axis_of)
            for h in range(src.shape[1]):
                want, size = rs.norm_rotate(src[i, h], weight, 1e-6, angles, interleaved)
                bound = (HALF_STEP[dtype] * np.abs(want) + 16 * 2.0 ** -24 * size) * (1 + 2.0 ** -7)
                assert (np.abs(got[i, h] - want) <= bound).all(), (t, h, float((np.abs(got[i, h] - want) - bound).max()))
