"""GPU parity of the rotary cache write against its fp64 definition.

Tolerances: the last step of an element adds two products in fp32; the norm
before it (a sum of head_dim squares whose tree is at most 8 + 4 additions
deep, one rsqrtf of 2 ulp, a multiply by 1/D, an addition, two multiplies) and
the rotation (two roundings) are each within a few 2^-24, together under 16
steps of 2^-24 of |y1 c| + |y2 s|.  The store rounds once: 2^-8 of the value
for bf16, 2^-24 for fp32.  Values are copied bit for bit.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import rope_sparse as rs

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_355_b200 as pa

    assert torch.cuda.is_available()
    pa.pa_read_error_flag()  # clear
    return pa


def f64(t):
    return t.detach().cpu().double().numpy()


def angle_table(last, rotary):
    freq = 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) * 2 / rotary)
    a = torch.arange(last, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


class Case:
    """Inputs of one call on the CPU: `tokens` new tokens, their slots distinct
    and scattered, every `skip`-th one padding."""

    def __init__(self, tokens, hq, hkv, d, bs, dtype, rotary, norm=(True, True), axes=1, skip=0, seed=0, last=200):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])
        self.dtype, self.tokens, self.bs, self.d = dtype, tokens, bs, d
        self.nb = tokens // bs + 4
        qkv = rnd(max(tokens, 1), hq + 2 * hkv, d)[:tokens]
        self.qkv, self.hq, self.hkv = qkv, hq, hkv
        self.k_pool, self.v_pool = rnd(self.nb, hkv, bs, d), rnd(self.nb, hkv, bs, d)
        self.query_out = rnd(tokens, hq, d)
        self.slots = torch.randperm(self.nb * bs, generator=g)[:tokens].to(torch.int64)
        if skip:
            self.slots[::skip] = -1
        self.positions = torch.randint(0, last, (axes, tokens), generator=g, dtype=torch.int32)
        self.pair_axes = torch.randint(0, axes, (rotary // 2,), generator=g, dtype=torch.int32) if axes > 1 else None
        self.cos_sin = angle_table(last, rotary)
        self.q_weight = (1 + 0.1 * torch.randn(d, generator=g)).to(DT[dtype]) if norm[0] else None
        self.k_weight = (1 + 0.1 * torch.randn(d, generator=g)).to(DT[dtype]) if norm[1] else None

    def split(self, t):
        return t[:, : self.hq], t[:, self.hq: self.hq + self.hkv], t[:, self.hq + self.hkv:]

    def want(self, slots=None, positions=None, interleaved=False, eps=1e-6):
        """fp64 arrays after the call, and each element's size (0: untouched)."""
        out, kp, vp = f64(self.query_out), f64(self.k_pool), f64(self.v_pool)
        q, k, v = self.split(f64(self.qkv))
        w = [None if x is None else f64(x) for x in (self.q_weight, self.k_weight)]
        qs, ks = rs.rope_and_cache(q, k, v, (self.slots if slots is None else slots).tolist(),
                                   (self.positions if positions is None else positions).numpy(), f64(self.cos_sin),
                                   None if self.pair_axes is None else self.pair_axes.numpy(), interleaved, w[0], w[1],
                                   eps, out, kp, vp)
        return out, kp, vp, qs, ks

    def check(self, query_out, k_pool, v_pool, **kw):
        out, kp, vp, qs, ks = self.want(**kw)
        for got, ref, size, what in ((query_out, out, qs, "query"), (k_pool, kp, ks, "key")):
            err = np.abs(f64(got) - ref)
            assert np.isfinite(err).all(), what
            bound = np.where(size > 0, HALF_STEP[self.dtype] * np.abs(ref) + 16 * 2.0 ** -24 * size, 0.0)
            # the rounding at the store is of the computed value
            bound = bound * (1 + 2.0 ** -7)
            bad = err > bound
            assert not bad.any(), f"{what}: {int(bad.sum())} elements off, worst {float((err - bound).max()):.3e}"
        assert np.array_equal(f64(v_pool), vp)


def call(pa, c, interleaved=False, **kw):
    qkv = c.qkv.cuda()
    q, k, v = c.split(qkv)
    out, kp, vp = c.query_out.cuda(), c.k_pool.cuda(), c.v_pool.cuda()
    cuda = lambda t: None if t is None else t.cuda()
    pa.pa_rope_and_cache(q, k, v, out, kp, vp, c.slots.cuda(), c.positions.cuda(), c.cos_sin.cuda(),
                         pair_axes=cuda(c.pair_axes), interleaved=interleaved, q_weight=cuda(c.q_weight),
                         k_weight=cuda(c.k_weight), eps=1e-6, **kw)
    torch.cuda.synchronize()
    return out, kp, vp


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,rotary", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [(True, True), (False, True), (True, False), (False, False)])
def test_prompt_rows(pa, dtype, d, rotary, interleaved, norm):
    c = Case(23, 8, 2, d, 16, dtype, rotary, norm, skip=7, seed=d + rotary)
    c.check(*call(pa, c, interleaved), interleaved=interleaved)
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("tokens,hq,hkv", [(1, 1, 1), (1, 32, 8), (3, 5, 5), (2, 7, 1), (64, 14, 4), (700, 12, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bs", [8, 32])
def test_head_counts_and_lengths(pa, tokens, hq, hkv, dtype, bs):
    """Odd head counts (a warp's last step is in part empty, q, k and v rows of
    one step mixed) and enough tokens for several steps a warp."""
    for d in (64, 128):
        c = Case(tokens, hq, hkv, d, bs, dtype, 32, skip=5 if tokens > 4 else 0, seed=tokens + hq)
        c.check(*call(pa, c))
    assert pa.pa_read_error_flag() == 0


def test_many_tokens_take_the_longest_unrolled_steps(pa):
    """9000 tokens of 24 head rows: 16 steps a warp and more than one warp a token."""
    c = Case(9000, 16, 4, 64, 16, "bf16", 64, (False, False), seed=3)
    out, kp, vp = call(pa, c)
    some = torch.arange(0, 9000, 97)
    slots = torch.full_like(c.slots, -1)
    slots[some] = c.slots[some]
    ref, rk, rv, qs, ks = c.want(slots=slots)
    touched = qs > 0
    assert (np.abs(f64(out) - ref)[touched] <= (1.01 * 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * qs)[touched]).all()
    touched = ks > 0
    assert (np.abs(f64(kp) - rk)[touched] <= (1.01 * 2.0 ** -8 * np.abs(rk) + 2.0 ** -20 * ks)[touched]).all()
    assert np.array_equal(f64(vp)[touched], rv[touched])
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_three_axes(pa, interleaved, dtype):
    c = Case(31, 4, 2, 128, 16, dtype, 96, axes=3, skip=9, seed=8)
    c.check(*call(pa, c, interleaved), interleaved=interleaved)
    # the same position on every axis is the one-axis call, bit for bit
    c.positions = c.positions[:1].expand(3, -1).contiguous()
    three = call(pa, c, interleaved)
    c.positions, c.pair_axes = c.positions[:1].contiguous(), None
    one = call(pa, c, interleaved)
    assert all(torch.equal(a, b) for a, b in zip(three, one))
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("given", [False, True])
def test_decode_form(pa, dtype, bs, given):
    """Slots from the table, an empty sequence, positions from the lengths or given."""
    B = 37
    c = Case(B, 8, 2, 128, bs, dtype, 128, seed=bs, last=400)
    g = torch.Generator().manual_seed(9)
    mbs = 5
    c.nb = B * mbs + 2
    c.k_pool = torch.randn(c.nb, 2, bs, 128, generator=g).to(DT[dtype])
    c.v_pool = torch.randn(c.nb, 2, bs, 128, generator=g).to(DT[dtype])
    tables = torch.randperm(c.nb, generator=g)[: B * mbs].reshape(B, mbs).to(torch.int32)
    lens = torch.randint(1, mbs * bs + 1, (B,), generator=g, dtype=torch.int32)
    lens[4], lens[5], lens[6] = 0, mbs * bs, 1
    at = (lens.long() - 1).clamp(min=0)
    slots = tables.gather(1, (at // bs)[:, None])[:, 0].long() * bs + at % bs
    slots[4] = -1
    positions = c.positions if given else (lens - 1)[None]
    out, kp, vp = c.query_out.cuda(), c.k_pool.cuda(), c.v_pool.cuda()
    got = torch.full((B,), 7, dtype=torch.int64, device="cuda")
    q, k, v = c.split(c.qkv.cuda())
    args = (q, k, v, out, kp, vp, tables.cuda(), lens.cuda(), c.cos_sin.cuda())
    kw = dict(positions=positions.cuda() if given else None, q_weight=c.q_weight.cuda(), k_weight=c.k_weight.cuda())
    pa.pa_rope_and_cache_decode(*args, **kw, slot_mapping=got)
    c.check(out, kp, vp, slots=slots, positions=positions)
    assert got.tolist() == slots.tolist()
    # without the slots output, and once more over its own result: the same bits
    again = [out.clone(), kp.clone(), vp.clone()]
    pa.pa_rope_and_cache_decode(*args, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, (out, kp, vp)))
    # the prompt form at the same slots and positions: the same bits
    c.slots, c.positions = slots, positions.clamp(min=0).to(torch.int32)
    assert all(torch.equal(a, b) for a, b in zip(again, call(pa, c)))
    assert pa.pa_read_error_flag() == 0


def test_layouts(pa):
    """Contiguous q, k and v, slices of one projection, and q rotated in place
    give the same bits; tokens further apart than a row need."""
    c = Case(19, 6, 2, 64, 16, "bf16", 64, seed=4)
    ref = call(pa, c)
    q, k, v = (t.contiguous().cuda() for t in c.split(c.qkv))
    rest = (c.slots.cuda(), c.positions.cuda(), c.cos_sin.cuda())
    w = dict(q_weight=c.q_weight.cuda(), k_weight=c.k_weight.cuda())
    out, kp, vp = c.query_out.cuda(), c.k_pool.cuda(), c.v_pool.cuda()
    pa.pa_rope_and_cache(q, k, v, out, kp, vp, *rest, **w)
    assert all(torch.equal(a, b) for a, b in zip(ref, (out, kp, vp)))
    kp, vp = c.k_pool.cuda(), c.v_pool.cuda()
    pa.pa_rope_and_cache(q, k, v, q, kp, vp, *rest, **w)
    assert all(torch.equal(a, b) for a, b in zip(ref, (q, kp, vp)))
    wide = torch.full((19, 14, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :10] = c.qkv.cuda()
    out, kp, vp = c.query_out.cuda(), c.k_pool.cuda(), c.v_pool.cuda()
    pa.pa_rope_and_cache(*c.split(wide[:, :10]), out, kp, vp, *rest, **w)
    assert all(torch.equal(a, b) for a, b in zip(ref, (out, kp, vp)))
    with pytest.raises(ValueError, match="heads of a token"):
        pa.pa_rope_and_cache(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, out, kp, vp, *rest, **w)
    assert pa.pa_read_error_flag() == 0


def test_token_strides_of_whole_vectors_only(pa):
    c = Case(3, 2, 1, 64, 16, "bf16", 64, seed=4)
    odd = torch.zeros(3, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, : 4 * 64].view(3, 4, 64)
    out, kp, vp = c.query_out.cuda(), c.k_pool.cuda(), c.v_pool.cuda()
    with pytest.raises(pa.PAError, match="PA_ERR_INVALID_ARG"):  # 520 bytes between tokens
        pa.pa_rope_and_cache(*c.split(odd), out, kp, vp, c.slots.cuda(), c.positions.cuda(), c.cos_sin.cuda())
    with pytest.raises(TypeError, match="k_pool must be torch.bfloat16"):
        pa.pa_rope_and_cache(*c.split(c.qkv.cuda()), out, kp.float(), vp, c.slots.cuda(), c.positions.cuda(),
                             c.cos_sin.cuda())
    with pytest.raises(TypeError, match="cos_sin must be torch.float32"):
        pa.pa_rope_and_cache(*c.split(c.qkv.cuda()), out, kp, vp, c.slots.cuda(), c.positions.cuda(),
                             c.cos_sin.cuda().double())
    with pytest.raises(TypeError, match="slot_mapping must be a CUDA tensor"):
        pa.pa_rope_and_cache(*c.split(c.qkv.cuda()), out, kp, vp, c.slots, c.positions.cuda(), c.cos_sin.cuda())
    assert torch.equal(kp.cpu(), c.k_pool)
    # one token may lie anywhere, and positions may be one row
    one = Case(1, 2, 1, 64, 16, "bf16", 64, seed=8)
    row = torch.zeros(1, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, : 4 * 64].view(1, 4, 64)
    row.copy_(one.qkv)
    out, kp, vp = one.query_out.cuda(), one.k_pool.cuda(), one.v_pool.cuda()
    pa.pa_rope_and_cache(*one.split(row), out, kp, vp, one.slots.cuda(), one.positions[0].cuda(), one.cos_sin.cuda(),
                         q_weight=one.q_weight.cuda(), k_weight=one.k_weight.cuda())
    one.check(out, kp, vp)
    assert pa.pa_read_error_flag() == 0


def test_no_tokens_and_far_positions(pa):
    c = Case(0, 4, 2, 64, 16, "f32", 64)
    before = c.k_pool.clone()
    out, kp, vp = call(pa, c)
    assert torch.equal(kp.cpu(), before)
    # the last row of a table of a million positions
    c = Case(5, 4, 2, 64, 16, "f32", 64, last=1_000_001, seed=2)
    c.positions[:] = 1_000_000
    c.check(*call(pa, c))
    assert pa.pa_read_error_flag() == 0


@pytest.mark.parametrize("what", ["slot", "position", "negative position", "axis"])
def test_bad_tokens_are_skipped_whole_and_flagged(pa, what):
    c = Case(9, 5, 3, 64, 16, "f32", 64, axes=2, seed=6)
    slots = c.slots.clone()
    if what == "slot":
        c.slots[4] = c.nb * 16
        slots[4] = -1
    elif what == "axis":
        c.pair_axes[3] = 2
        slots[:] = -1  # every token uses every pair
    else:
        c.positions[1, 4] = 200 if what == "position" else -1
        c.pair_axes[5] = 1
        slots[4] = -1
    got = call(pa, c)
    c.positions, c.pair_axes = c.positions.clamp(0, 199), c.pair_axes.clamp(max=1)
    c.check(*got, slots=slots)
    assert pa.pa_read_error_flag() == 5
    assert pa.pa_read_error_flag() == 0


def test_bad_sequences_of_the_decode_form(pa):
    c = Case(5, 4, 2, 64, 8, "f32", 64, (False, False), seed=7)
    tables = torch.tensor([[0], [-1], [c.nb], [1], [2]], dtype=torch.int32)
    lens = torch.tensor([3, 2, 2, 9, -4], dtype=torch.int32)  # unmapped, past the pool, past the table, negative
    out, kp, vp = c.query_out.cuda(), c.k_pool.cuda(), c.v_pool.cuda()
    got = torch.full((5,), 7, dtype=torch.int64, device="cuda")
    pa.pa_rope_and_cache_decode(*c.split(c.qkv.cuda()), out, kp, vp, tables.cuda(), lens.cuda(), c.cos_sin.cuda(),
                                slot_mapping=got)
    slots = torch.tensor([2, -1, -1, -1, -1])
    assert got.tolist() == slots.tolist()
    c.check(out, kp, vp, slots=slots, positions=(lens - 1)[None].clamp(min=0))
    assert pa.pa_read_error_flag() == 5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_elements_stay_in_their_pair(pa, dtype):
    """An infinity past the rotated part, or in one pair, leaves the rest alone."""
    c = Case(2, 2, 1, 64, 16, dtype, 32, (False, False), seed=5)
    for interleaved in (False, True):
        clean = call(pa, c, interleaved)[0]
        c.qkv[0, 0, 40] = float("inf")
        c.qkv[1, 1, 3] = float("inf")
        out = call(pa, c, interleaved)[0]
        assert out[0, 0, 40] == float("inf")
        out[0, 0, 40] = clean[0, 0, 40]
        touched = [2, 3] if interleaved else [3, 19]
        assert not out[1, 1, touched].isfinite().any()
        out[1, 1, touched] = clean[1, 1, touched]
        assert torch.equal(out, clean)
        c = Case(2, 2, 1, 64, 16, dtype, 32, (False, False), seed=5)


def test_nan_rows_stay_in_their_head(pa):
    """A NaN in one head, and in a padded token, reaches no other row."""
    c = Case(6, 4, 2, 128, 16, "bf16", 128, seed=5)
    clean = call(pa, c)
    c.slots[2] = -1
    skipped = call(pa, c)
    c.qkv[2] = float("nan")
    assert all(torch.equal(a, b) for a, b in zip(skipped, call(pa, c)))
    c.qkv[3, 1] = float("nan")
    out, kp, vp = call(pa, c)
    assert out[3, 1].isnan().all() and torch.equal(kp, skipped[1]) and torch.equal(vp, skipped[2])
    out[3, 1] = skipped[0][3, 1]
    assert torch.equal(out, skipped[0]) and not clean[0].isnan().any()
    assert pa.pa_read_error_flag() == 0


def test_streams_and_graphs(pa):
    """On another stream than the current one, and replayed from a graph over
    new inputs in the same buffers."""
    c = Case(33, 8, 2, 128, 16, "bf16", 128, seed=1)
    ref = call(pa, c)
    side = torch.cuda.Stream()
    got = call(pa, c, stream=side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    qkv, out, kp, vp = c.qkv.cuda(), c.query_out.cuda(), c.k_pool.cuda(), c.v_pool.cuda()
    rest = (c.slots.cuda(), c.positions.cuda(), c.cos_sin.cuda())
    w = dict(q_weight=c.q_weight.cuda(), k_weight=c.k_weight.cuda())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rope_and_cache(*c.split(qkv), out, kp, vp, *rest, **w)
    for seed in (1, 11):
        d = Case(33, 8, 2, 128, 16, "bf16", 128, seed=seed)
        qkv.copy_(d.qkv)
        out.copy_(d.query_out)
        kp.copy_(d.k_pool)
        vp.copy_(d.v_pool)
        rest[0].copy_(d.slots)
        rest[1].copy_(d.positions)
        w["q_weight"].copy_(d.q_weight)
        w["k_weight"].copy_(d.k_weight)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(call(pa, d), (out, kp, vp)))
    assert pa.pa_read_error_flag() == 0
