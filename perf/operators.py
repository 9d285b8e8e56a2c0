"""The cache, page-selection and draft-tree operators of the MLA decode library, as cases to measure.

Each case is one call as a serving program makes it; ``run`` computes it in plain torch (``own`` false) or
through the library (``own`` true).  Shapes: latent rows of 512 dims and 64 RoPE dims (d = 576) or 512 dims alone
(d = 512), pages of 64 tokens, bf16 pages or packed e4m3 pages with per-token scales.

  write   rows of new tokens into the pages of their sequences (e4m3: quantised per token)
  read    rows of a range of each sequence back to contiguous bf16 rows (e4m3: dequantised)
  keys    the int8 key of every page that a sequence's new tokens touched
  blocks  decode over the pages that a score against the page keys selects for each query token
  tree    decode of a tree of drafted tokens whose rows end each sequence
"""
import math

import torch

own = False

PAGE, DV, ROPE = 64, 512, 64


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token per sequence: what every decoding step writes in every layer; latency counts
        {"name": "write_bf16_step", "op": "write", "fp8": False, "d": 576, "b": 64, "lo": 1, "hi": 1, "past": 2048, "pad": 0},
        # prompts of many lengths written at once into an e4m3 cache, the input buffer padded behind them
        {"name": "write_fp8_prompt", "op": "write", "fp8": True, "d": 576, "b": 8, "lo": 1500, "hi": 8192, "past": 2048, "pad": 77},
        # a chunk of the prompt path reads its whole cached context back for the up-projection
        {"name": "read_fp8_context", "op": "read", "fp8": True, "d": 576, "b": 16, "lo": 256, "hi": 8192, "past": 512, "pad": 0},
        # a short ragged range of a cache of 512-wide rows
        {"name": "read_bf16_d512", "op": "read", "fp8": False, "d": 512, "b": 5, "lo": 0, "hi": 333, "past": 700, "pad": 19},
        # a decoding step touches the last page of each sequence
        {"name": "keys_bf16_step", "op": "keys", "fp8": False, "d": 576, "b": 64, "lo": 1, "hi": 8, "past": 4096, "pad": 0},
        # after the prompts: the keys of every page
        {"name": "keys_fp8_prompt", "op": "keys", "fp8": True, "d": 576, "b": 16, "lo": 1000, "hi": 16384, "past": 0, "pad": 0},
        # one request with few heads: latency
        {"name": "blocks_bf16_small", "op": "blocks", "fp8": False, "d": 576, "b": 1, "s": 1, "h": 16, "lo": 3500, "hi": 3500, "top": 8, "causal": False},
        # multi-token steps over an e4m3 cache of ragged lengths
        {"name": "blocks_fp8_mtp", "op": "blocks", "fp8": True, "d": 576, "b": 16, "s": 4, "h": 128, "lo": 500, "hi": 16384, "top": 24, "causal": True},
        # the long decode (64 sequences of 65,536 tokens), one sixteenth of the pages attended to
        {"name": "blocks_bf16_long", "op": "blocks", "fp8": False, "d": 576, "b": 64, "s": 1, "h": 128, "lo": 65536, "hi": 65536, "top": 64, "causal": False},
        # a small tree of drafts for one request with few heads
        {"name": "tree_bf16_small", "op": "tree", "fp8": False, "d": 576, "b": 1, "s": 8, "h": 16, "lo": 500, "hi": 500},
        # ragged trees over an e4m3 cache, 13 nodes at most, 64 heads
        {"name": "tree_fp8_ragged", "op": "tree", "fp8": True, "d": 576, "b": 24, "s": 13, "h": 64, "lo": 256, "hi": 8192},
        # trees of 32 nodes at all 128 heads over long ragged contexts: bound by the tensor cores
        {"name": "tree_bf16_large", "op": "tree", "fp8": False, "d": 576, "b": 16, "s": 32, "h": 128, "lo": 2048, "hi": 8192},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "keys", "blocks", "blocks", "tree", "tree"])
    fp8 = rng.random() < 0.5
    d = 576 if fp8 or rng.random() < 0.7 else 512
    if op in ("write", "read", "keys"):
        b = _spread(rng, 1, 128)
        hi = _spread(rng, 1, min(8192, 65536 // b))
        return {"op": op, "fp8": fp8, "d": d, "b": b, "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi,
                "past": rng.randint(0, 2048), "pad": rng.choice([0, 0, 1, rng.randint(2, 100)]) if op != "keys" else 0}
    if op == "blocks":
        b, s = _spread(rng, 1, 48), rng.choice([1, 1, 1, 2, 3, 4, 8])
        hi = _spread(rng, 1, min(65536, (1 << 20) // (b * s)))
        top = _spread(rng, 3, 64)
        return {"op": op, "fp8": fp8, "d": d, "b": b, "s": s, "h": rng.choice([16, 32, 64, 128, 128, rng.randint(1, 160)]),
                "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi, "top": top, "causal": rng.random() < 0.7}
    s, h = _spread(rng, 1, 64), rng.choice([16, 32, 64, 128, 128, rng.randint(1, 160)])
    b = _spread(rng, 1, 32)
    hi = _spread(rng, 1, max(1, min(16384, (1 << 28) // (b * s * h))))
    return {"op": op, "fp8": fp8, "d": d, "b": b, "s": s, "h": h, "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi}


# ---------------------------------------------------------------- inputs
def _pages_of(rows):
    """Packed e4m3 pages of fp32 rows [n, 64, 576]: 64 rows of codes, then 64 fp32 scales."""
    n, _, d = rows.shape
    amax = rows.abs().amax(-1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), 1.0)
    pages = torch.empty((n, PAGE * d + PAGE * 4), dtype=torch.uint8, device=rows.device)
    pages[:, :PAGE * d] = (rows / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(n, PAGE * d)
    pages[:, PAGE * d:] = scale.view(torch.uint8).reshape(n, PAGE * 4)
    return pages


def _random_cache(g, nblk, d, fp8, dev):
    """A pool whose pages have a subject of their own: every row is its page's direction plus its own noise."""
    out = torch.empty((nblk, PAGE * d + PAGE * 4), dtype=torch.uint8, device=dev) if fp8 else \
        torch.empty((nblk, PAGE, 1, d), dtype=torch.bfloat16, device=dev)
    topic = torch.randn((nblk, 1, d), generator=g, device=dev) * 0.6
    for lo in range(0, nblk, 4096):
        rows = torch.randn((min(4096, nblk - lo), PAGE, d), generator=g, device=dev).mul_(0.8).add_(topic[lo:lo + 4096])
        out[lo:lo + 4096] = _pages_of(rows) if fp8 else rows.to(torch.bfloat16)[:, :, None]
    return out


def _ancestors(parent):
    """Which nodes node i sees, [b, s, s]: itself and its ancestors (parent < i, or -1 for a root)."""
    b, s = parent.shape
    at = torch.arange(s)
    sees = torch.eye(s, dtype=torch.bool).repeat(b, 1, 1)
    for i in range(s):
        up = sees[torch.arange(b), parent[:, i].clamp(min=0)] & (parent[:, i] >= 0)[:, None]
        sees[:, i] |= up & (at < i)
    return sees


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    gc = torch.Generator()
    gc.manual_seed(seed)
    op, d, b = case["op"], case["d"], case["b"]
    # the lengths are the case's own, so that buffers have one size; what lies where and what it holds is the seed's
    count = torch.randint(case["lo"], case["hi"] + 1, (b,), generator=torch.Generator().manual_seed(7 * b + case["hi"]))
    if op in ("write", "read", "keys"):
        start = torch.randint(0, case["past"] + 1, (b,), generator=gc)
    else:
        start = torch.zeros((b,), dtype=torch.int64)
        count[0] = case["hi"]  # the longest is always there
    if op == "tree":
        nodes = torch.randint(max(1, case["s"] // 2), case["s"] + 1, (b,), generator=gc)
        nodes[0] = case["s"]
        count = count.clamp(min=case["s"])
    length = start + count
    need = (length + PAGE - 1) // PAGE
    most = (count + case.get("past", 0) + PAGE - 1) // PAGE
    width = max(1, int(most.max()))
    nblk = int(most.sum()) + 3
    table = torch.zeros((b, width), dtype=torch.int64)
    used = torch.arange(width)[None] < need[:, None]
    table[used] = torch.randperm(nblk, generator=gc)[:int(need.sum())]
    to = lambda t: t.to(torch.int32).to(dev)  # noqa: E731
    state = {"case": case, "op": op, "d": d, "b": b, "fp8": case["fp8"], "dev": dev, "table": to(table),
             "lens": to(length), "cache": _random_cache(g, nblk, d, case["fp8"], dev)}
    if op in ("write", "read"):
        cu = torch.zeros((b + 1,), dtype=torch.int64)
        cu[1:] = count.cumsum(0)
        n = max(1, int(cu[-1]) + case["pad"])
        state |= {"starts": to(start), "cu": to(cu), "n": n}
        # both parts as slices of one projection's output, or as the buffers that the read fills
        both = torch.randn((n, d), generator=g, device=dev).to(torch.bfloat16) if op == "write" else \
            torch.zeros((n, d), dtype=torch.bfloat16, device=dev)
        state |= {"latent": both[:, :DV], "rope": both[:, DV:] if d > DV else None}
    elif op == "keys":
        state |= {"starts": to(start), "keys": torch.zeros((nblk, d), dtype=torch.int8, device=dev),
                  "scales": torch.zeros((nblk,), device=dev)}
    else:
        q = torch.randn((b, case["s"], case["h"], d), generator=g, device=dev)
        state |= {"q": (1.5 * q).to(torch.bfloat16), "softmax_scale": d ** -0.5}
        if op == "blocks":
            rows = _rows(state, state["cache"])
            state["keys"], state["scales"] = _key_of(rows, torch.full((nblk,), float(PAGE), device=dev))
            del rows
        else:
            parent = torch.stack([torch.randint(max(-1, i - 5), i, (b,), generator=gc) if i else torch.full((b,), -1)
                                  for i in range(case["s"])], 1)
            sees = _ancestors(parent)
            words = (case["s"] + 31) // 32
            bits = torch.nn.functional.pad(sees, (0, 32 * words - case["s"])).view(b, case["s"], words, 32)
            packed = (bits.to(torch.int64) << torch.arange(32)).sum(-1)
            packed = torch.where(packed >= 1 << 31, packed - (1 << 32), packed)
            state |= {"mask": to(packed), "nodes": to(nodes)}
    return state


# ---------------------------------------------------------------- plain forms
def _codes(state, pages):
    """The pages' codes [n, 64, d] and scales [n, 64], as views."""
    d = state["d"]
    return (pages[:, :PAGE * d].view(torch.float8_e4m3fn).unflatten(1, (PAGE, d)),
            pages[:, PAGE * d:].view(torch.float32))


def _rows(state, pages):
    """fp32 rows [n, 64, d] of pages."""
    if state["fp8"]:
        codes, scales = _codes(state, pages)
        return codes.float() * scales[..., None]
    return pages.flatten(1).unflatten(1, (PAGE, state["d"])).float()


def _place(state):
    """For every row behind cu: (is it of a sequence, its physical block, its row in the page)."""
    r = torch.arange(state["n"], device=state["dev"])
    cu = state["cu"].long()
    seq = (r[:, None] >= cu[None, 1:]).sum(1)
    live = seq < state["b"]
    seq = seq.clamp(max=state["b"] - 1)
    pos = torch.where(live, state["starts"].long()[seq] + r - cu[seq], 0)
    return live, state["table"].long()[seq, pos // PAGE], pos % PAGE


def _write(state):
    live, blk, off = _place(state)
    x = state["latent"] if state["rope"] is None else torch.cat([state["latent"], state["rope"]], 1)
    x, blk, off = x[live], blk[live], off[live]
    if not state["fp8"]:
        state["cache"][blk, off, 0] = x
        return state["cache"]
    x = x.float()
    amax = x.abs().amax(1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), 1.0)  # by a tensor: the quotient itself
    codes, scales = _codes(state, state["cache"])
    codes.view(torch.uint8)[blk, off] = (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scales[blk, off] = scale
    return [codes, scales]


def _read(state):
    live, blk, off = _place(state)
    if state["fp8"]:
        codes, scales = _codes(state, state["cache"])
        x = (codes.view(torch.uint8)[blk, off].view(torch.float8_e4m3fn).float() * scales[blk, off][:, None]).bfloat16()
    else:
        x = state["cache"][blk, off, 0]
    state["latent"][live] = x[live, :DV]
    if state["rope"] is not None:
        state["rope"][live] = x[live, DV:]
    return [state["latent"], state["rope"]]


def _key_of(rows, count):
    """int8 keys and their scales for the means of rows [n, 64, d] (absent rows 0), summed two by two."""
    x = rows[:, 0::2] + rows[:, 1::2]
    x = x[:, 0::2] + x[:, 1::2]
    x = x[:, 0::2] + x[:, 1::2]
    x = x[:, 0::2] + x[:, 1::2]
    x = x[:, 0::2] + x[:, 1::2]
    mean = (x[:, 0] + x[:, 1]) / count[:, None]
    amax = mean.abs().amax(1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 127.0), 1.0)
    return torch.round(mean / scale[:, None]).to(torch.int8), scale


def _keys(state):
    page = torch.arange(state["table"].shape[1], device=state["dev"])[None]
    lens, first = state["lens"].long()[:, None], state["starts"].long()[:, None] // PAGE
    touched = (page >= first) & (page * PAGE < lens)
    blk = state["table"].long()[touched]
    count = (lens - page * PAGE).clamp(max=PAGE)[touched]
    there = torch.arange(PAGE, device=state["dev"])[None] < count[:, None]
    rows = torch.where(there[..., None], _rows(state, state["cache"][blk]), 0.0)
    state["keys"][blk], state["scales"][blk] = _key_of(rows, count.float())
    return [state["keys"], state["scales"]]


def _attend(q, rows, seen, scale):
    """Softmax attention of q [.., r, d] over rows [.., t, d] where seen [.., r, t]; a row that sees nothing gives 0."""
    z = torch.where(seen, torch.matmul(q.float(), rows.transpose(-1, -2)) * scale, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows[..., :DV]) / torch.where(total > 0, total, 1.0)
    return o.bfloat16(), (torch.log(total) + top)[..., 0]


def _blocks(state):
    case, q, table = state["case"], state["q"], state["table"].long()
    b, s, h, d = q.shape
    width, top, dev = table.shape[1], case["top"], state["dev"]
    amax = q.float().abs().amax(-1, keepdim=True)
    qs = torch.where(amax > 0, amax / torch.full_like(amax, 127.0), 1.0)
    qi = torch.round(q.float() / qs)
    dots = torch.matmul(qi.view(b, s * h, d), state["keys"][table].float().transpose(1, 2)).view(b, s, h, width)
    score = (dots * qs).amax(2) * state["scales"][table][:, None]
    back = torch.arange(s - 1, -1, -1, device=dev) if case["causal"] else torch.zeros((s,), dtype=torch.long, device=dev)
    ends = (state["lens"].long()[:, None] - back).clamp(min=0)  # [b, s]
    count = (ends + PAGE - 1) // PAGE
    page = torch.arange(width, device=dev)
    score = torch.where((page < 1) | (page == count[..., None] - 1), math.inf, score)
    score = torch.where(page < count[..., None], score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    if width < top:
        best = torch.nn.functional.pad(best, (0, top - width), value=width)
    best = torch.where(best < count[..., None], best, width).sort(-1).values  # ascending, absent ones behind
    there = best < width
    blk = torch.gather(table[:, None].expand(b, s, width), 2, best.clamp(max=width - 1))
    rows = _rows(state, state["cache"][blk.view(-1)]).view(b, s, top * PAGE, d)
    pos = best[..., None] * PAGE + torch.arange(PAGE, device=dev)
    seen = (there[..., None] & (pos < ends[..., None, None])).view(b, s, 1, top * PAGE)
    rows = torch.where(seen.transpose(-1, -2), rows, 0.0)
    o, lse = _attend(q, rows, seen, state["softmax_scale"])
    return [o, lse, torch.where(there, best, -1).to(torch.int32)]


def _tree(state):
    q, table, dev = state["q"], state["table"].long(), state["dev"]
    b, s, h, d = q.shape
    t = table.shape[1] * PAGE
    pos = torch.arange(t, device=dev)
    lens, nodes = state["lens"].long(), state["nodes"].long()
    node = pos - (lens - nodes)[:, None]  # [b, t]
    there = pos < lens[:, None]
    rows = _rows(state, state["cache"][table.view(-1)]).view(b, t, d)
    rows = torch.where(there[..., None], rows, 0.0)
    at = node.clamp(0, s - 1)[:, None].expand(b, s, t)
    bit = (torch.gather(state["mask"].long(), 2, at // 32) >> (at % 32)) & 1
    seen = there[:, None] & ((node < 0)[:, None] | (bit == 1)) & (torch.arange(s, device=dev)[:, None] < nodes[:, None, None])
    seen = seen[:, :, None].expand(b, s, h, t).reshape(b, s * h, t)
    o, lse = _attend(q.view(b, s * h, d), rows, seen, state["softmax_scale"])
    return [o.view(b, s, h, DV), lse.view(b, s, h)]


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if own:
        import mla_decode_attention_latent_gb300 as mla
        fp8, cache, table = state["fp8"], state["cache"], state["table"]
        if op == "write":
            write = mla.mla_cache_write_fp8 if fp8 else mla.mla_cache_write
            write(state["latent"], state["rope"], cache, table, state["starts"], cu_rows=state["cu"])
            return list(_codes(state, cache)) if fp8 else cache
        if op == "read":
            read = mla.mla_cache_read_fp8 if fp8 else mla.mla_cache_read
            read(cache, table, state["starts"], state["n"], cu_rows=state["cu"], latent=state["latent"], k_rope=state["rope"])
            return [state["latent"], state["rope"]]
        if op == "keys":
            update = mla.mla_update_page_keys_fp8 if fp8 else mla.mla_update_page_keys
            update(cache, table, state["lens"], state["keys"], state["scales"], starts=state["starts"])
            return [state["keys"], state["scales"]]
        if op == "blocks":
            decode = mla.mla_decode_kvcache_blocks_fp8 if fp8 else mla.mla_decode_kvcache_blocks
            return list(decode(state["q"], cache, table, state["lens"], state["keys"], state["scales"], state["case"]["top"], DV,
                               softmax_scale=state["softmax_scale"], causal=state["case"]["causal"]))
        decode = mla.mla_decode_kvcache_tree_fp8 if fp8 else mla.mla_decode_kvcache_tree
        return list(decode(state["q"], cache, table, state["lens"], state["mask"], DV, tree_lens=state["nodes"],
                           softmax_scale=state["softmax_scale"]))
    return {"write": _write, "read": _read, "keys": _keys, "blocks": _blocks, "tree": _tree}[op](state)


def _mean(case):
    return (case["lo"] + case["hi"]) / 2.0


def work(case):
    op, d, b = case["op"], case["d"], case["b"]
    row = d + 4 if case["fp8"] else 2 * d  # bytes of a cached row
    n = _mean(case) * b
    if op in ("write", "read"):
        return {"bytes": max(1.0, n) * (2 * d + row), "flops": max(1.0, n) * d * (2 if case["fp8"] else 0)}
    if op == "keys":
        pages = b * (_mean(case) / PAGE + 0.5)
        return {"bytes": max(n, b * PAGE / 2.0) * row + pages * (d + 4), "flops": max(n, 1.0) * d}
    s, h = case["s"], case["h"]
    rows = b * s * h
    io = rows * (2 * d + 2 * DV + 4)
    if op == "blocks":
        t = max(1.0, _mean(case))
        pages = math.ceil(t / PAGE)
        top = min(pages, case["top"])
        return {"bytes": io + b * (pages * (d + 4) + min(pages, top * s) * PAGE * row),
                "flops": 2.0 * rows * (pages * d + min(t, top * PAGE) * (d + DV))}
    t = max(_mean(case), 0.75 * s)
    return {"bytes": io + b * t * row, "flops": 2.0 * 0.75 * rows * t * (d + DV)}


# ---------------------------------------------------------------- in 64 bits
def _f32(x):
    """Round to 32 bits, where the operator's definition does."""
    return x.to(torch.float32).double()


def _row64(state, blk, off):
    """One cached row after another, in 64 bits."""
    d, cache = state["d"], state["cache"]
    if not state["fp8"]:
        return cache.view(-1, d)[blk * PAGE + off].double()
    flat = cache.view(torch.float8_e4m3fn).view(-1)
    at = blk[:, None] * cache.shape[1] + off[:, None] * d + torch.arange(d, device=cache.device)
    scale = cache.view(torch.float32)[blk, PAGE * d // 4 + off]
    return flat.view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * scale.double()[:, None]


def _sequence(state, b, lo, hi):
    """Blocks and rows of positions lo .. hi - 1 of sequence b."""
    pos = torch.arange(lo, hi, device=state["dev"])
    return state["table"][b].long()[pos // PAGE], pos % PAGE


def exact(case, seed):
    state = prepare(case, seed)
    op, d = state["op"], state["d"]
    if op in ("write", "read"):
        cu, starts = state["cu"].tolist(), state["starts"].tolist()
        if op == "write":
            x = (state["latent"] if state["rope"] is None else torch.cat([state["latent"], state["rope"]], 1)).double()
            if state["fp8"]:
                codes, scales = [t.double() for t in _codes(state, state["cache"])]
            else:
                rows = state["cache"].double()
        else:
            lat = state["latent"].double()
            rope = None if state["rope"] is None else state["rope"].double()
        for b in range(state["b"]):
            lo, hi = cu[b], cu[b + 1]
            blk, off = _sequence(state, b, starts[b], starts[b] + hi - lo)
            if op == "read":
                got = _row64(state, blk, off)
                lat[lo:hi] = got[:, :DV]
                if rope is not None:
                    rope[lo:hi] = got[:, DV:]
            elif state["fp8"]:
                big = x[lo:hi].abs().max(1).values if hi > lo else x[lo:hi, 0]
                c = _f32(torch.where(big > 0, big / torch.full_like(big, 448), torch.ones_like(big)))
                scales[blk, off] = c
                codes[blk, off] = (x[lo:hi] / c[:, None]).float().to(torch.float8_e4m3fn).double()
            else:
                rows[blk, off, 0] = x[lo:hi]
        return [lat, rope] if op == "read" else [codes, scales] if state["fp8"] else rows
    if op == "keys":
        keys, scales = torch.zeros_like(state["keys"]), state["scales"].double()
        starts, lens = state["starts"].tolist(), state["lens"].tolist()
        for b in range(state["b"]):
            first, pages = starts[b] // PAGE, -(-lens[b] // PAGE)
            if pages <= first:
                continue
            blk, off = _sequence(state, b, first * PAGE, lens[b])
            rows = torch.zeros(((pages - first) * PAGE, d), dtype=torch.float64, device=state["dev"])
            rows[:blk.numel()] = _f32(_row64(state, blk, off))
            x, n = rows.view(pages - first, PAGE, d), PAGE
            while n > 1:  # the definition's order: neighbours first, each sum in 32 bits
                n //= 2
                x = _f32(x.view(pages - first, n, 2, d).sum(2))
            size = torch.full((pages - first, 1), float(PAGE), dtype=torch.float64, device=state["dev"])
            size[-1] = lens[b] - (pages - 1) * PAGE
            mean = _f32(x[:, 0] / size)
            big = mean.abs().max(1, keepdim=True).values
            c = _f32(torch.where(big > 0, big / torch.full_like(big, 127), torch.ones_like(big)))
            keys[state["table"][b].long()[first:pages]] = _f32(mean / c).round().to(torch.int8)
            scales[state["table"][b].long()[first:pages]] = c[:, 0]
        return [keys, scales]
    q = state["q"].double()
    b, s, h, _ = q.shape
    lens = state["lens"].tolist()
    if 2.0 * b * s * h * max(lens) * (d + DV) > 2e13:
        return None
    o = torch.zeros((b, s, h, DV), dtype=torch.float64, device=state["dev"])
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64, device=state["dev"])
    chosen = torch.full((b, s, case.get("top", 1)), -1, dtype=torch.int32, device=state["dev"])
    for i in range(b):
        if op == "tree":
            nodes = int(state["nodes"][i])
            base = lens[i] - nodes
            rows = _row64(state, *_sequence(state, i, 0, lens[i]))
            words = state["mask"][i].tolist()
        for j in range(s):
            if op == "tree":
                if j >= nodes:
                    continue
                seen = [base + k for k in range(nodes) if base + k >= 0 and (words[j][k // 32] >> (k % 32)) & 1]
                keys = rows[torch.tensor(list(range(max(0, base))) + seen, dtype=torch.long, device=state["dev"])]
            else:
                end = lens[i] - (s - 1 - j if case["causal"] else 0)
                if end <= 0:
                    continue
                pages = -(-end // PAGE)
                if pages <= case["top"]:
                    pick = list(range(pages))
                else:
                    big = q[i, j].abs().max(1, keepdim=True).values
                    unit = _f32(torch.where(big > 0, big / torch.full_like(big, 127), torch.ones_like(big)))
                    whole = _f32(q[i, j] / unit).round()
                    blk = state["table"][i, :pages].long()
                    each = _f32((whole @ state["keys"][blk].double().T) * unit).max(0).values
                    each = _f32(each * state["scales"][blk].double()).tolist()
                    rest = sorted(range(1, pages - 1), key=lambda p: (-each[p], p))[:case["top"] - 2]
                    pick = sorted([0, pages - 1] + rest)
                chosen[i, j, :len(pick)] = torch.tensor(pick, dtype=torch.int32, device=state["dev"])
                pos = (torch.tensor(pick, device=state["dev"])[:, None] * PAGE + torch.arange(PAGE, device=state["dev"])).view(-1)
                pos = pos[pos < end]
                keys = _row64(state, state["table"][i].long()[pos // PAGE], pos % PAGE)
            if not keys.shape[0]:
                continue
            z = q[i, j] @ keys.T * state["softmax_scale"]
            lse[i, j] = torch.logsumexp(z, 1)
            o[i, j] = torch.exp(z - lse[i, j][:, None]) @ keys[:, :DV]
    return [o, lse] if op == "tree" else [o, lse, chosen]
