"""Refusals of the rotary cache write and the block-sparse calls, on the host:
the C entry points return before any launch, and the binding names what is
wrong.  No GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
P, I64, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_355_b200 import build

    return ctypes.CDLL(build.build())


def _rope(lib, decode=False, **kw):
    a = dict(q=16, k=16, v=16, qs=1024, ks=256, vs=256, qo=16, kp=16, vp=16, slots=16, bt=16, mbs=4, lens=16, pos=16,
             axes=1, pair=0, cs=16, maxpos=100, rot=64, inter=0, qw=0, kw=0, eps=1e-6, T=5, hq=8, hkv=2, d=128, bs=16,
             nb=10, dt=1)
    a.update(kw)
    head = (P(a["q"]), P(a["k"]), P(a["v"]), I64(a["qs"]), I64(a["ks"]), I64(a["vs"]), P(a["qo"]), P(a["kp"]),
            P(a["vp"]))
    tail = (P(a["pos"]), a["axes"], P(a["pair"]), P(a["cs"]), I64(a["maxpos"]), a["rot"], a["inter"], P(a["qw"]),
            P(a["kw"]), F(a["eps"]))
    sizes = (a["hq"], a["hkv"], a["d"], a["bs"], I64(a["nb"]), a["dt"])
    if decode:
        return lib.pa_rope_and_cache_decode(*head, P(a["bt"]), a["mbs"], P(a["lens"]), *tail, a["T"], *sizes, P(0), None)
    return lib.pa_rope_and_cache(*head, P(a["slots"]), *tail, I64(a["T"]), *sizes, None)


@pytest.mark.parametrize("decode", [False, True])
def test_rope_refusals(lib, decode):
    bad = lambda **kw: _rope(lib, decode, **kw)
    assert bad(T=0, q=0, kp=0) == OK                 # nothing to do, nothing launched
    for name in ("q", "k", "v", "qo", "kp", "vp", "cs"):
        assert bad(**{name: 0}) == INVALID
        assert bad(**{name: 24}) == INVALID          # not 16-byte aligned
    assert bad(qw=24) == INVALID and bad(kw=8) == INVALID
    assert bad(qs=1023) == INVALID                   # less than a row
    assert bad(qs=1028) == INVALID                   # not a multiple of 16 bytes
    assert bad(ks=255) == INVALID and bad(vs=250) == INVALID
    assert bad(d=96) == UNSUPPORTED
    assert bad(bs=64) == UNSUPPORTED
    for rot in (0, 8, 24, 136, -16):
        assert bad(rot=rot) == UNSUPPORTED
    assert bad(inter=2) == INVALID
    assert bad(dt=5) == INVALID
    assert bad(eps=-1.0) == INVALID and bad(eps=float("nan")) == INVALID
    assert bad(axes=0) == INVALID
    assert bad(axes=3) == INVALID                    # several axes need pair_axes
    assert bad(maxpos=0) == INVALID                  # no table row
    assert bad(T=-1) == INVALID and bad(hq=0) == INVALID and bad(hkv=0) == INVALID
    if not decode:
        assert bad(T=1 << 40) == UNSUPPORTED
    if decode:
        assert bad(bt=0) == INVALID and bad(lens=0) == INVALID
        assert bad(pos=0, axes=3, pair=16) == INVALID
        assert bad(pos=0, pair=16) == INVALID
    else:
        assert bad(slots=0) == INVALID and bad(pos=0) == INVALID


def _bounds(lib, **kw):
    a = dict(k=16, kb=16, bt=16, mbs=4, lens=16, qs=0, maxq=1, B=2, hkv=2, d=128, bs=16, nb=10, dt=1)
    a.update(kw)
    return lib.pa_update_key_bounds(P(a["k"]), P(a["kb"]), P(a["bt"]), a["mbs"], P(a["lens"]), P(a["qs"]), a["maxq"],
                                    a["B"], a["hkv"], a["d"], a["bs"], I64(a["nb"]), a["dt"], None)


def test_bounds_refusals(lib):
    assert _bounds(lib, B=0, k=0) == OK
    assert _bounds(lib, qs=16, maxq=0) == OK         # no new token anywhere
    assert _bounds(lib, maxq=0) == INVALID
    assert _bounds(lib, maxq=-1, qs=16) == INVALID
    for name in ("k", "kb", "bt", "lens"):
        assert _bounds(lib, **{name: 0}) == INVALID
    assert _bounds(lib, k=24) == INVALID and _bounds(lib, kb=24) == INVALID
    assert _bounds(lib, d=32) == UNSUPPORTED and _bounds(lib, bs=4) == UNSUPPORTED
    assert _bounds(lib, dt=2) == INVALID and _bounds(lib, B=-1) == INVALID


def _scores(lib, **kw):
    a = dict(q=16, kb=16, bt=16, mbs=4, seq=0, lens=16, maxlen=50, bs=16, sc=16, stride=4, R=2, B=2, hq=8, hkv=2,
             d=128, nb=10, dt=1)
    a.update(kw)
    return lib.pa_block_scores(P(a["q"]), P(a["kb"]), P(a["bt"]), a["mbs"], P(a["seq"]), P(a["lens"]), a["maxlen"],
                               a["bs"], P(a["sc"]), I64(a["stride"]), I64(a["R"]), a["B"], a["hq"], a["hkv"], a["d"],
                               I64(a["nb"]), a["dt"], None)


def test_scores_refusals(lib):
    assert _scores(lib, R=0, q=0) == OK
    for name in ("q", "kb", "bt", "lens", "sc"):
        assert _scores(lib, **{name: 0}) == INVALID
    assert _scores(lib, q=24) == INVALID
    assert _scores(lib, maxlen=65) == INVALID        # longer than the table can map
    assert _scores(lib, stride=3) == INVALID         # fewer columns than blocks
    assert _scores(lib, R=3) == INVALID              # more rows than sequences, no seq_ids
    assert _scores(lib, hq=7) == INVALID
    assert _scores(lib, hq=6) == UNSUPPORTED         # group of 3
    assert _scores(lib, hq=32, dt=0) == UNSUPPORTED  # group of 16 needs bf16
    assert _scores(lib, d=96) == UNSUPPORTED and _scores(lib, bs=64) == UNSUPPORTED
    assert _scores(lib, R=1 << 60, seq=16) == UNSUPPORTED
    assert _scores(lib, maxlen=-1) == INVALID and _scores(lib, dt=9) == INVALID


def _select(lib, **kw):
    a = dict(sc=16, stride=4, lens=16, maxlen=50, bs=16, sel=16, K=4, first=1, last=2, R=2, hkv=2)
    a.update(kw)
    return lib.pa_select_blocks(P(a["sc"]), I64(a["stride"]), P(a["lens"]), a["maxlen"], a["bs"], P(a["sel"]), a["K"],
                                a["first"], a["last"], I64(a["R"]), a["hkv"], None)


def test_select_refusals(lib):
    assert _select(lib, R=0, sc=0) == OK
    for name in ("sc", "lens", "sel"):
        assert _select(lib, **{name: 0}) == INVALID
    assert _select(lib, K=2) == INVALID              # fewer than the blocks always taken
    assert _select(lib, K=0, first=0, last=0) == INVALID
    assert _select(lib, first=-1) == INVALID and _select(lib, last=-1) == INVALID
    assert _select(lib, first=2**31 - 1, last=2**31 - 1) == INVALID
    assert _select(lib, stride=3) == INVALID
    assert _select(lib, bs=12) == UNSUPPORTED
    assert _select(lib, R=1 << 60) == UNSUPPORTED
    assert _select(lib, hkv=0) == INVALID and _select(lib, R=-1) == INVALID


def _sparse(lib, **kw):
    a = dict(q=16, k=16, v=16, bt=16, mbs=4, seq=0, lens=16, sel=16, K=4, scale=0.1, bs=16, out=16, odt=0, R=2, B=2,
             hq=8, hkv=2, d=128, nb=10, dt=1)
    a.update(kw)
    return lib.pa_paged_attention_decode_sparse(
        P(a["q"]), P(a["k"]), P(a["v"]), P(a["bt"]), a["mbs"], P(a["seq"]), P(a["lens"]), P(a["sel"]), a["K"],
        F(a["scale"]), a["bs"], P(a["out"]), a["odt"], I64(a["R"]), a["B"], a["hq"], a["hkv"], a["d"], I64(a["nb"]),
        a["dt"], None)


def test_sparse_decode_refusals(lib):
    assert _sparse(lib, R=0, q=0) == OK
    for name in ("q", "k", "v", "bt", "lens", "sel", "out"):
        assert _sparse(lib, **{name: 0}) == INVALID
    for name in ("q", "k", "v", "out"):
        assert _sparse(lib, **{name: 24}) == INVALID
    assert _sparse(lib, K=0) == INVALID
    assert _sparse(lib, R=3) == INVALID
    assert _sparse(lib, hq=7) == INVALID and _sparse(lib, hq=6) == UNSUPPORTED
    assert _sparse(lib, hq=32, dt=0) == UNSUPPORTED
    assert _sparse(lib, d=80) == UNSUPPORTED and _sparse(lib, bs=1) == UNSUPPORTED
    assert _sparse(lib, R=1 << 60, seq=16) == UNSUPPORTED
    assert _sparse(lib, odt=2) == INVALID and _sparse(lib, dt=2) == INVALID


def test_binding_names_what_is_wrong(lib):
    """Shapes, layouts, types and places that the binding refuses by name."""
    import paged_kv_cache_355_b200 as pa

    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    q, kv, pool = z(3, 4, 64), z(3, 2, 64), z(5, 2, 16, 64)
    i32 = torch.int32
    lens, tables, cs = z(3, dtype=i32), z(3, 2, dtype=i32), z(10, 64)
    with pytest.raises(TypeError, match="query must be a CUDA tensor"):
        pa.pa_rope_and_cache_decode(q, kv, kv, q, pool, pool, tables, lens, cs)
    with pytest.raises(ValueError, match="shapes disagree"):
        pa.pa_rope_and_cache_decode(q, kv, kv, z(3, 5, 64), pool, pool, tables, lens, cs)
    with pytest.raises(TypeError, match="unsupported element type"):
        pa.pa_rope_and_cache_decode(q.half(), kv, kv, q, pool, pool, tables, lens, cs)
    with pytest.raises(ValueError, match="key_bounds must be"):
        pa.pa_update_key_bounds(pool, z(5, 2, 64), tables, lens)
    with pytest.raises(ValueError, match="query_start batch"):
        pa.pa_update_key_bounds(pool, z(5, 2, 2, 64), tables, lens, query_start=z(3, dtype=i32))
    with pytest.raises(ValueError, match="shapes disagree"):
        pa.pa_block_scores(q, z(5, 2, 2, 64), tables, lens, 20, 16, z(3, 3, 2))
    with pytest.raises(ValueError, match="shapes disagree"):
        pa.pa_select_blocks(z(3, 2, 2), lens, 20, 16, z(3, 2, dtype=i32))
    with pytest.raises(ValueError, match="selected must be"):
        pa.pa_paged_attention_decode_sparse(q, pool, pool, tables, lens, z(3, 4, 2, dtype=i32), 0.1, q)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        pa.pa_paged_attention_decode_sparse(q, pool, pool, tables, lens, z(3, 2, 2, dtype=i32), 0.1, q)


def test_marshalling_signatures_are_the_entry_points(lib):
    """The C module's letters, argument by argument, against the ctypes types,
    and a name for every tensor it may refuse."""
    from paged_kv_cache_355_b200 import _binding as b

    scalar = {"I": b._I, "L": b._I64, "F": b._F}
    assert len(b._ENTRIES) == 6
    for name, signature in b._ENTRIES:
        types, _ = b._SIGS[name]
        assert [scalar.get(c, b._P) for c in signature] == types, name
        names = b._ARG_NAMES[name].split()
        assert all(i < len(names) for i, c in enumerate(signature) if c in "KilforkjmR"), name
    order = (b._ROPE, b._ROPE_DECODE, b._BOUNDS, b._SCORES, b._SELECT, b._SPARSE)
    assert [b._ENTRIES[i][0] for i in order] == [
        "pa_rope_and_cache", "pa_rope_and_cache_decode", "pa_update_key_bounds", "pa_block_scores", "pa_select_blocks",
        "pa_paged_attention_decode_sparse"]


def test_marshalling_refuses(lib):
    from paged_kv_cache_355_b200 import _binding as b

    call = b._marshal.call
    with pytest.raises(TypeError, match="wrong number of arguments"):
        call(b._SELECT, 0, None, ())
    with pytest.raises(ValueError, match="no such entry point"):
        call(6, 0, None, ())
    with pytest.raises(ValueError, match="no such entry point"):
        call(-1, 0, None, ())
    with pytest.raises(TypeError):
        call(b._SELECT, 0, None, [])
    # what is no tensor, or a tensor on the CPU, is refused by its place
    for t in (None, 3, "x", torch.zeros(2)):
        assert call(b._SELECT, 0, None, (t,) * 12) == -1
        assert call(b._SELECT, -1, None, (t,) * 12) == -1
