"""Cases of the rotary cache write and of block-sparse decode attention, for timing and comparison.

Five calls make one decode step that attends to a chosen part of a long context:

  append   head norms of q and k, the rotation of positions, and the write of k and v into the paged cache
  bounds   per block and channel, the smallest and the largest key value
  scores   for each query row, kv head and block, an upper bound of the block's dot products with the queries
  select   the blocks that a row's kv head attends to: the first, the last, and those of the largest score
  attend   softmax attention over the tokens of the selected blocks

``run`` computes them with elementary torch operations where ``own`` is false and through the
package's entry points where it is true; ``exact`` computes them in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(name, form, seqs, lo, hi, hq, hkv, d, bs, dtype, norm, axes, interleaved, rotary, pad=0, lens=1):
    """form "decode": one token for each of seqs sequences of lo..hi tokens; form "prompt": seqs prompts of
    lo..hi tokens, and `pad` padding tokens behind them."""
    return {"name": name, "op": "append", "form": form, "seqs": seqs, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d,
            "bs": bs, "dtype": dtype, "norm": norm, "axes": axes, "interleaved": interleaved, "rotary": rotary,
            "pad": pad, "lens": lens}


def _sparse(name, op, seqs, lo, hi, hq, hkv, d, bs, dtype, budget=0, rows=1, pad=0, lens=1):
    """seqs sequences of lo..hi tokens, the last `pad` of them empty; `rows` query rows (its last tokens) a
    sequence; budget: blocks attended to at most."""
    return {"name": name, "op": op, "seqs": seqs, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d, "bs": bs,
            "dtype": dtype, "budget": budget, "rows": rows, "pad": pad, "lens": lens}


def listed():
    return [
        # the smallest decode step: four short sequences in fp32, where only the call's latency counts
        _append("append decode batch 4", "decode", 4, 2, 34, 4, 4, 64, 16, "f32", False, 1, False, 64),
        # an ordinary decode step with grouped heads and head norms
        _append("append decode batch 256", "decode", 256, 16, 1024, 32, 8, 128, 16, "bf16", True, 1, False, 128),
        # prompts of one prefill chunk, every query head with its own kv head, half of each head rotated
        _append("append prompts 8k tokens", "prompt", 7, 128, 2048, 32, 32, 128, 16, "bf16", False, 1, True, 64),
        # a long prompt of images and text: three position axes, head norms, and a padded tail
        _append("append images 24k tokens", "prompt", 3, 7000, 9000, 64, 8, 128, 32, "bf16", True, 3, False, 128, 61),
        # the summary of each sequence's last block after a decode step
        _sparse("bounds decode batch 64", "bounds", 64, 128, 2048, 32, 32, 128, 16, "bf16"),
        # the summaries of whole prompts after their prefill (rows 0: every token is new)
        _sparse("bounds prompts", "bounds", 8, 16384, 65536, 64, 8, 128, 16, "bf16", rows=0),
        # block scores of a large batch of ordinary lengths
        _sparse("scores batch 256", "scores", 256, 16, 4096, 32, 8, 128, 16, "bf16", pad=3),
        # block scores of long contexts
        _sparse("scores long", "scores", 16, 32768, 131072, 64, 8, 128, 16, "bf16"),
        # the choice for a large batch, and for long contexts
        _sparse("select batch 256", "select", 256, 16, 4096, 32, 8, 128, 16, "bf16", 64, pad=3),
        _sparse("select long", "select", 16, 32768, 131072, 64, 8, 128, 16, "bf16", 256),
        # one long conversation: few rows, so the work has to be split over the blocks
        _sparse("attend one sequence", "attend", 1, 32768, 32768, 32, 8, 128, 16, "bf16", 128),
        # long contexts, 4096 tokens attended to of up to 131072
        _sparse("attend long", "attend", 16, 32768, 131072, 64, 8, 128, 16, "bf16", 256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "bounds", "scores", "select", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d, bs = rng.choice([64, 128]), rng.choice([8, 16, 32])
    hkv = rng.choice([1, 2, 4, 5, 8])
    hq = hkv * rng.choice([1, 2, 4, 8, 16] if dtype == "bf16" else [1, 2, 4, 8])
    lens = rng.randrange(1, 1 << 20)
    while True:
        if op == "append":
            form = rng.choice(["decode", "prompt"])
            axes = rng.choice([1, 1, 3])
            rotary = rng.choice([16, 32, 64, d])
            if form == "decode":
                case = _append("", form, _log(rng, 1, 256), 1, _log(rng, 16, 1024), hq, hkv, d, bs, dtype,
                               rng.random() < 0.5, axes, rng.random() < 0.5, rotary, 0, lens)
            else:
                hi = _log(rng, 8, 8192)
                case = _append("", form, rng.randint(1, 6), rng.randint(1, hi), hi, hq, hkv, d, bs, dtype,
                               rng.random() < 0.5, axes, rng.random() < 0.5, rotary, rng.choice([0, 0, 7]), lens)
        else:
            hi = _log(rng, 100, 131072)
            case = _sparse("", op, _log(rng, 1, 256), rng.randint(1, hi), hi, hq, hkv, d, bs, dtype,
                           _log(rng, 8, 512) if op in ("select", "attend") else 0,
                           rng.choice([0, 1]) if op == "bounds" else rng.choice([1, 1, 1, 3]), 0, lens)
            case["pad"] = min(case["seqs"] - 1, rng.choice([0, 0, 2]))
        tokens = case["seqs"] * (case["hi"] + bs)
        # the cache of a drawn case takes 4 GiB at most, and the pass 300 MB
        if tokens * hkv * d * (2 if dtype == "bf16" else 4) * 2 <= 4 << 30 and work(case)["bytes"] <= 300_000_000:
            del case["name"]
            return case


def _lengths(case):
    """Tokens of each sequence: the same for every seed, so that work() can count them."""
    r, lo, hi = random.Random(case["lens"]), case["lo"], case["hi"]
    n, pad = case["seqs"], case["pad"] if case["op"] != "append" else 0
    out = [r.randint(lo, hi) if hi <= 8 * lo else _log(r, lo, hi) for _ in range(n)]
    return out[: n - pad] + [0] * pad


def _rows(case):
    """(sequence, length seen) of every query row: the last tokens of each sequence."""
    n = case["rows"]
    return [(b, max(0, L - (n - 1 - i))) for b, L in enumerate(_lengths(case)) for i in range(n)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _device_lengths(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _tables(lengths, bs, gen):
    """Each sequence's blocks, scattered over a pool that is a tenth larger than needed."""
    need = [-(-L // bs) for L in lengths]
    total = sum(need)
    nb = total + total // 10 + 1
    ids = torch.randperm(nb, generator=gen, device="cuda", dtype=torch.int32)
    width = max(1, max(need))
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col[None, :]).clamp_(max=nb - 1)
    tables = torch.where(col[None, :] < torch.tensor(need, device="cuda")[:, None], ids[at], -1)
    return tables.to(torch.int32).contiguous(), nb


def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _keys(shape, dtype, gen):
    """Keys with channels of unequal size and offset, as projections give them (the last axis is the channel)."""
    d = shape[-1]
    size = torch.exp(torch.randn(d, generator=gen, device="cuda") * 0.5).to(dtype)
    offset = torch.randn(d, generator=gen, device="cuda").to(dtype)
    return _normal(shape, dtype, gen).mul_(size).add_(offset)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    lengths = _lengths(case)
    s = dict(case, scale=1.0 / math.sqrt(d), max_len=max(lengths), context_lens=_device_lengths(lengths))
    if case["op"] == "append":
        return _prepare_append(s, case, lengths, dtype, gen)
    s["block_tables"], nb = _tables(lengths, bs, gen)
    if case["op"] == "bounds":
        s["k_pool"] = _keys((nb, hkv, bs, d), dtype, gen)
        s["key_bounds"] = torch.zeros((nb, hkv, 2, d), dtype=dtype, device="cuda")
        if case["rows"] == 0:
            starts = [0]
            for L in lengths:
                starts.append(starts[-1] + L)
            s["query_start"] = _device_lengths(starts)
        return s
    rows = _rows(case)
    s["seq_ids"] = None if case["rows"] == 1 else _device_lengths([b for b, _ in rows])
    s["context_lens"] = _device_lengths([L for _, L in rows])
    n, blocks = len(rows), s["block_tables"].shape[1]
    if case["op"] != "select":
        s["q"] = _normal((n, hq, d), dtype, gen)
    if case["op"] == "scores":
        a, b = _keys((nb, hkv, d), dtype, gen), _normal((nb, hkv, d), dtype, gen).abs_()
        s["key_bounds"] = torch.stack([a - b, a + b], dim=2)
        s["scores"] = torch.zeros((n, hkv, blocks), device="cuda")
        return s
    if case["op"] == "select":
        # scores around a common level, on a grid, so that some are equal
        level = torch.randn((n, hkv, blocks), generator=gen, device="cuda") * 12 + 60
        s["scores"] = torch.round(level * 64) / 64
        s["selected"] = torch.zeros((n, hkv, case["budget"]), dtype=torch.int32, device="cuda")
        return s
    s["k_pool"] = _keys((nb, hkv, bs, d), dtype, gen)
    s["v_pool"] = _normal((nb, hkv, bs, d), dtype, gen)
    # a choice in ascending order with the last block in it, -1 behind it
    have = (s["context_lens"] + bs - 1) // bs
    col = torch.arange(blocks, device="cuda")
    chance = torch.rand((n, hkv, blocks), generator=gen, device="cuda")
    chance = torch.where(col == have[:, None, None] - 1, 2.0, chance)
    chance = torch.where(col < have[:, None, None], chance, -1.0)
    k = min(case["budget"], blocks)
    top, at = chance.topk(k, dim=2)
    at = torch.where(top >= 0, at, blocks).sort(dim=2).values
    selected = torch.full((n, hkv, case["budget"]), -1, dtype=torch.int32, device="cuda")
    selected[:, :, :k] = torch.where(at < blocks, at, -1)
    s["selected"] = selected
    s["out"] = torch.zeros((n, hq, d), dtype=dtype, device="cuda")
    return s


def _prepare_append(s, case, lengths, dtype, gen):
    hq, hkv, d, bs, axes, rotary = (case[k] for k in ("hq", "hkv", "d", "bs", "axes", "rotary"))
    decode = case["form"] == "decode"
    tables, nb = _tables(lengths, bs, gen)
    tokens = len(lengths) if decode else sum(lengths) + case["pad"]
    # one projection gives q, k and v: three views of its rows
    qkv = _normal((tokens, hq + 2 * hkv, d), dtype, gen)
    s["query"], s["key"], s["value"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["query_out"] = torch.zeros((tokens, hq, d), dtype=dtype, device="cuda")
    s["k_pool"] = _normal((nb, hkv, bs, d), dtype, gen)
    s["v_pool"] = _normal((nb, hkv, bs, d), dtype, gen)
    s["q_weight"] = (_normal((d,), dtype, gen) * 0.1 + 1) if case["norm"] else None
    s["k_weight"] = (_normal((d,), dtype, gen) * 0.1 + 1) if case["norm"] else None
    last = max(lengths)
    frequency = 10000.0 ** (-torch.arange(rotary // 2, device="cuda", dtype=torch.float64) * 2 / rotary)
    angle = torch.arange(last, device="cuda", dtype=torch.float64)[:, None] * frequency
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    if decode:
        s["block_tables"] = tables
        s["seq"] = torch.arange(len(lengths), device="cuda")
        text = s["context_lens"] - 1
    else:
        seq = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths)).cuda()
        text = torch.cat([torch.arange(L) for L in lengths]).to(torch.int32).cuda()
        slots = tables[seq, text // bs].long() * bs + text % bs
        pad = torch.full((case["pad"],), -1, device="cuda")
        s["slot_mapping"] = torch.cat([slots, pad])
        text = torch.cat([text, torch.zeros(case["pad"], dtype=torch.int32, device="cuda")])
    if axes == 1:
        s["positions"], s["pair_axes"] = text[None].contiguous(), None
    else:
        # a grid of 24 columns: time, height and width of each token, and the pairs shared out among them
        s["positions"] = torch.stack([text, text // 24 % 24, text % 24]).to(torch.int32).contiguous()
        s["pair_axes"] = (torch.arange(rotary // 2, device="cuda") % 3).to(torch.int32)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _own_append(s):
    import paged_kv_cache_355_b200 as pa

    if s["form"] == "decode":
        pa.pa_rope_and_cache_decode(s["query"], s["key"], s["value"], s["query_out"], s["k_pool"], s["v_pool"],
                                    s["block_tables"], s["context_lens"], s["cos_sin"],
                                    positions=None if s["axes"] == 1 else s["positions"],
                                    pair_axes=s["pair_axes"], interleaved=s["interleaved"], q_weight=s["q_weight"],
                                    k_weight=s["k_weight"], eps=1e-6)
    else:
        pa.pa_rope_and_cache(s["query"], s["key"], s["value"], s["query_out"], s["k_pool"], s["v_pool"],
                             s["slot_mapping"], s["positions"], s["cos_sin"], pair_axes=s["pair_axes"],
                             interleaved=s["interleaved"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6)
    return {"query": s["query_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _own_bounds(s):
    import paged_kv_cache_355_b200 as pa

    if s["rows"] == 0:
        pa.pa_update_key_bounds(s["k_pool"], s["key_bounds"], s["block_tables"], s["context_lens"],
                                query_start=s["query_start"], max_query_len=s["max_len"])
    else:
        pa.pa_update_key_bounds(s["k_pool"], s["key_bounds"], s["block_tables"], s["context_lens"])
    return {"key_bounds": s["key_bounds"]}


def _own_scores(s):
    import paged_kv_cache_355_b200 as pa

    pa.pa_block_scores(s["q"], s["key_bounds"], s["block_tables"], s["context_lens"], s["max_len"], s["bs"],
                       s["scores"], seq_ids=s["seq_ids"])
    return {"scores": s["scores"]}


def _own_select(s):
    import paged_kv_cache_355_b200 as pa

    pa.pa_select_blocks(s["scores"], s["context_lens"], s["max_len"], s["bs"], s["selected"], num_first=1, num_last=2)
    return {"selected": s["selected"]}


def _own_attend(s):
    import paged_kv_cache_355_b200 as pa

    pa.pa_paged_attention_decode_sparse(s["q"], s["k_pool"], s["v_pool"], s["block_tables"], s["context_lens"],
                                        s["selected"], s["scale"], s["out"], seq_ids=s["seq_ids"])
    return {"out": s["out"]}


def _norm_rotate(x, weight, c, sn, rotary, interleaved):
    """x [T, H, D] in 32 bits; c, sn [T, rotary / 2]."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * weight.float()
    turned, rest = x[..., :rotary], x[..., rotary:]
    c, sn = c[:, None], sn[:, None]
    if interleaved:
        x1, x2 = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([x1 * c - x2 * sn, x2 * c + x1 * sn], dim=-1).flatten(-2)
    else:
        x1, x2 = turned[..., :rotary // 2], turned[..., rotary // 2:]
        turned = torch.cat([x1 * c - x2 * sn, x2 * c + x1 * sn], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _plain_append(s):
    bs, rotary, dtype = s["bs"], s["rotary"], s["key"].dtype
    if s["form"] == "decode":
        text = s["context_lens"].long() - 1
        slots = s["block_tables"][s["seq"], text // bs].long() * bs + text % bs
    else:
        slots = s["slot_mapping"]
    keep = (slots >= 0).nonzero()[:, 0]
    slots = slots[keep]
    pair = torch.arange(rotary // 2, device="cuda")
    axis = s["pair_axes"].long() if s["pair_axes"] is not None else torch.zeros_like(pair)
    at = s["positions"][:, keep].long()[axis]                         # [pair, token]
    c, sn = s["cos_sin"][at, pair[:, None]].T, s["cos_sin"][at, rotary // 2 + pair[:, None]].T
    q = _norm_rotate(s["query"][keep].float(), s["q_weight"], c, sn, rotary, s["interleaved"])
    k = _norm_rotate(s["key"][keep].float(), s["k_weight"], c, sn, rotary, s["interleaved"])
    s["query_out"][keep] = q.to(dtype)
    s["k_pool"][slots // bs, :, slots % bs] = k.to(dtype)
    s["v_pool"][slots // bs, :, slots % bs] = s["value"][keep]
    return {"query": s["query_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_bounds(s):
    bs, lens = s["bs"], s["context_lens"].long()
    new = lens if s["rows"] == 0 else (lens > 0).long()
    col = torch.arange(s["block_tables"].shape[1], device="cuda")
    touched = (col >= ((lens - new) // bs)[:, None]) & (col < ((lens + bs - 1) // bs)[:, None]) & (new > 0)[:, None]
    seq, block = touched.nonzero(as_tuple=True)
    phys = s["block_tables"][seq, block].long()
    k = s["k_pool"][phys].float()
    held = (block[:, None] * bs + torch.arange(bs, device="cuda") < lens[seq][:, None])[:, None, :, None]
    low = k.masked_fill(~held, float("inf")).amin(dim=2)
    high = k.masked_fill(~held, float("-inf")).amax(dim=2)
    s["key_bounds"][phys] = torch.stack([low, high], dim=2).to(s["k_pool"].dtype)
    return {"key_bounds": s["key_bounds"]}


def _row_tables(s):
    return s["block_tables"] if s["seq_ids"] is None else s["block_tables"][s["seq_ids"].long()]


def _plain_scores(s):
    n, hq, d = s["q"].shape
    hkv, bs = s["hkv"], s["bs"]
    tables, have = _row_tables(s), (s["context_lens"] + bs - 1) // bs
    bounds = s["key_bounds"][tables.clamp(min=0).long()].float()      # [rows, blocks, hkv, 2, d]
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    low, high = (bounds[:, :, :, i].permute(0, 2, 3, 1) for i in (0, 1))
    each = torch.matmul(q.clamp(min=0), high) + torch.matmul(q.clamp(max=0), low)
    held = torch.arange(tables.shape[1], device="cuda") < have[:, None, None]
    s["scores"] = torch.where(held, each.amax(dim=2), s["scores"])
    return {"scores": s["scores"]}


def _plain_select(s):
    budget, bs = s["budget"], s["bs"]
    scores, have = s["scores"], ((s["context_lens"] + bs - 1) // bs)[:, None, None]
    col = torch.arange(scores.shape[2], device="cuda")
    forced = (col < 1) | (col >= have - 2)
    rank = torch.where(col < have, torch.where(forced, float("inf"), scores), float("-inf"))
    at = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :budget]
    at = torch.where(at < have, at, scores.shape[2]).sort(dim=2).values
    s["selected"].fill_(-1)
    s["selected"][:, :, :at.shape[2]] = torch.where(at < scores.shape[2], at, -1)
    return {"selected": s["selected"]}


def _plain_attend(s):
    n, hq, d = s["q"].shape
    hkv, bs = s["hkv"], s["bs"]
    chosen = s["selected"].long()                                     # [rows, hkv, budget]
    tables = _row_tables(s)[:, None].expand(-1, hkv, -1)
    phys = torch.gather(tables, 2, chosen.clamp(min=0)).clamp(min=0).long()
    head = torch.arange(hkv, device="cuda")[None, :, None]
    k = s["k_pool"][phys, head].float().flatten(2, 3)                 # [rows, hkv, budget * bs, d]
    token = (chosen * bs)[..., None] + torch.arange(bs, device="cuda")
    seen = ((chosen >= 0)[..., None] & (token < s["context_lens"][:, None, None, None])).flatten(2)[:, :, None]
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    x = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).masked_fill(~seen, float("-inf"))
    del k
    top = x.amax(dim=3, keepdim=True)
    p = torch.exp(x - torch.where(top > float("-inf"), top, 0.0))
    v = s["v_pool"][phys, head].float().flatten(2, 3)
    total = p.sum(dim=3, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(out.view(n, hq, d))
    return {"out": s["out"]}


_OWN = {"append": _own_append, "bounds": _own_bounds, "scores": _own_scores, "select": _own_select,
        "attend": _own_attend}
_PLAIN = {"append": _plain_append, "bounds": _plain_bounds, "scores": _plain_scores, "select": _plain_select,
          "attend": _plain_attend}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e, hq, hkv, d, bs = 2 if case["dtype"] == "bf16" else 4, case["hq"], case["hkv"], case["d"], case["bs"]
    lengths = _lengths(case)
    if case["op"] == "append":
        tokens = len(lengths) if case["form"] == "decode" else sum(lengths)
        angles = min(tokens, max(lengths)) * case["rotary"] * 4
        return {"bytes": tokens * (2 * hq + 4 * hkv) * d * e + angles + tokens * 12,
                "flops": tokens * (hq + hkv) * (3 * case["rotary"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "bounds":
        if case["rows"] == 0:
            read, blocks = sum(lengths), sum(-(-L // bs) for L in lengths)
        else:
            read, blocks = sum((L - 1) % bs + 1 for L in lengths if L), sum(1 for L in lengths if L)
        return {"bytes": (read + 2 * blocks) * hkv * d * e + blocks * 4, "flops": 2 * read * hkv * d}
    rows = _rows(case)
    have = [-(-L // bs) for _, L in rows]
    distinct = sum(-(-L // bs) for L in lengths)
    if case["op"] == "scores":
        return {"bytes": distinct * (hkv * 2 * d * e + 4) + len(rows) * hq * d * e + sum(have) * hkv * 4,
                "flops": 4 * d * hq * sum(have)}
    if case["op"] == "select":
        return {"bytes": sum(have) * hkv * 4 + len(rows) * hkv * case["budget"] * 4, "flops": sum(have) * hkv}
    blocks = [min(h, case["budget"]) for h in have]
    held = [max(0, n * bs - (-L) % bs) for n, (_, L) in zip(blocks, rows)]
    read = min(sum(held), sum(lengths))
    return {"bytes": read * hkv * 2 * d * e + 2 * len(rows) * hq * d * e + len(rows) * hkv * case["budget"] * 4,
            "flops": 4 * d * hq * sum(held)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _exact_head(x, weight, angle_row, pair_axes, rotary, interleaved):
    """One projection's heads [T, H, D] in 64 bits; angle_row [axes, T, rotary]: the table rows of each axis."""
    x = x.double()
    if weight is not None:
        x = weight.double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
    out, half = x.clone(), rotary // 2
    for p in range(half):
        row = angle_row[pair_axes[p]]
        turn = torch.complex(row[:, p], row[:, half + p])[:, None]
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        z = torch.complex(x[..., a], x[..., b]) * turn
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_append(s):
    bs, rotary = s["bs"], s["rotary"]
    if s["form"] == "decode":
        pos = s["context_lens"].long().cpu() - 1
        table = s["block_tables"].cpu()
        slots = torch.tensor([int(table[b, int(p) // bs]) * bs + int(p) % bs for b, p in enumerate(pos)]).cuda()
    else:
        slots = s["slot_mapping"]
    real = slots >= 0
    rows = s["cos_sin"].double()[s["positions"].long()]
    axes = [0] * (rotary // 2) if s["pair_axes"] is None else s["pair_axes"].tolist()
    out = {"query": s["query_out"].double(), "k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
    q = _exact_head(s["query"], s["q_weight"], rows, axes, rotary, s["interleaved"])
    out["query"][real] = q[real]
    del q
    k = _exact_head(s["key"], s["k_weight"], rows, axes, rotary, s["interleaved"])
    nb, hkv, _, d = s["k_pool"].shape
    for name, x in (("k_pool", k), ("v_pool", s["value"].double())):
        flat = out[name].transpose(1, 2).reshape(nb * bs, hkv, d)
        flat[slots[real]] = x[real]
        out[name] = flat.view(nb, bs, hkv, d).transpose(1, 2).contiguous()
    return out


def _exact_bounds(s):
    bs, k, out = s["bs"], s["k_pool"], s["key_bounds"].double()
    tables, lens = s["block_tables"].cpu(), s["context_lens"].tolist()
    for b, L in enumerate(lens):
        if L == 0:
            continue
        first = 0 if s["rows"] == 0 else (L - 1) // bs
        full = tables[b, first: L // bs].long().cuda()
        if full.numel():
            whole = k[full].double()
            out[full] = torch.stack([whole.min(dim=2).values, whole.max(dim=2).values], dim=2)
        if L % bs:
            last = int(tables[b, L // bs])
            part = k[last, :, : L % bs].double()
            out[last] = torch.stack([part.min(dim=1).values, part.max(dim=1).values], dim=1)
    return {"key_bounds": out}


def _exact_scores(s):
    hkv, bs, out = s["hkv"], s["bs"], s["scores"].double()
    group = s["q"].shape[1] // hkv
    lens = s["context_lens"].tolist()
    seqs = list(range(len(lens))) if s["seq_ids"] is None else s["seq_ids"].tolist()
    for r, L in enumerate(lens):
        n = -(-L // bs)
        if n == 0:
            continue
        bounds = s["key_bounds"][s["block_tables"][seqs[r], :n].long()].double()     # [n, hkv, 2, d]
        for h in range(s["q"].shape[1]):
            q, g = s["q"][r, h].double(), h // group
            best = torch.maximum(bounds[:, g, 0] * q, bounds[:, g, 1] * q).sum(dim=1)
            out[r, g, :n] = best if h % group == 0 else torch.maximum(out[r, g, :n], best)
    return {"scores": out}


def _exact_select(s):
    import numpy as np

    scores, lens, bs, budget = s["scores"].cpu().numpy(), s["context_lens"].tolist(), s["bs"], s["budget"]
    out = np.full(s["selected"].shape, -1, np.int32)
    for r, L in enumerate(lens):
        n = -(-L // bs)
        always = {0} | set(range(max(0, n - 2), n)) if n else set()
        for g in range(scores.shape[1]):
            order = np.lexsort((np.arange(n), -scores[r, g, :n].astype(np.float64)))
            kept = sorted(always) + [j for j in order[: budget + 3].tolist() if j not in always]
            kept = sorted(kept[:budget])
            out[r, g, : len(kept)] = kept
    return {"selected": torch.from_numpy(out)}


def _exact_attend(s):
    n, hq, d = s["q"].shape
    hkv, bs = s["hkv"], s["bs"]
    group, lens = hq // hkv, s["context_lens"].tolist()
    seqs = list(range(n)) if s["seq_ids"] is None else s["seq_ids"].tolist()
    out = torch.zeros((n, hq, d), dtype=torch.float64, device="cuda")
    for r in range(n):
        for g in range(hkv):
            blocks = s["selected"][r, g].long()
            blocks = blocks[blocks >= 0]
            if blocks.numel() == 0:
                continue
            phys = s["block_tables"][seqs[r]].long()[blocks]
            at = (blocks[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)
            k, v = (s[p][phys, g].reshape(-1, d)[at < lens[r]].double() for p in ("k_pool", "v_pool"))
            x = s["q"][r, g * group:(g + 1) * group].double() @ k.T * s["scale"]
            out[r, g * group:(g + 1) * group] = torch.exp(x - torch.logsumexp(x, dim=1, keepdim=True)) @ v
    return {"out": out}


_EXACT = {"append": _exact_append, "bounds": _exact_bounds, "scores": _exact_scores, "select": _exact_select,
          "attend": _exact_attend}
