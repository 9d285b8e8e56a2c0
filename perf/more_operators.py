"""The prompt-path operators of the MLA decode library, as cases to measure.

Each case is one call as a serving program makes it; ``run`` computes it in plain torch (``own`` false) or
through the library (``own`` true).  Shapes: heads of 128 dims and 64 RoPE dims (a query head of 192), latent rows of
512 dims and 64 RoPE dims, pages of 64 tokens, bf16 pages or packed e4m3 pages with per-token scales.

  pages    block tables, positions and slots of the new rows of a step, pages taken from a free list
  rope     norm of every head and rotation of a part of it, in one pass
  place    norm of the latent rows, rotation of their RoPE keys, and the rows into the pages by slot
  prefill  attention of packed prompts (or chunks of them behind a context), causal or not, grouped heads
"""
import math

import torch

own = False

PAGE, LATENT, ROPE, HEAD = 64, 512, 64, 128
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token per sequence of a decoding batch: what every step begins with; latency counts
        {"name": "pages_step", "op": "pages", "b": 64, "lo": 1, "hi": 1, "past": 4096, "pad": 0, "short": False},
        # prompts of many lengths admitted at once, the row buffer padded behind them, more than the pool holds
        {"name": "pages_prompts", "op": "pages", "b": 48, "lo": 1, "hi": 4096, "past": 700, "pad": 77, "short": True},
        # a step's query heads: the rotated part goes from the projection's heads into the absorbed queries
        {"name": "rope_step", "op": "rope", "n": 64, "h": 128, "d": 64, "wide": 192, "out_wide": 576, "dims": 64, "norm": False, "interleaved": True,
         "factor": 40.0},
        # query and key heads that are normalised one by one, the whole head rotated, an odd number of tokens
        {"name": "rope_heads", "op": "rope", "n": 1777, "h": 40, "d": 128, "wide": 128, "out_wide": 128, "dims": 128, "norm": True, "interleaved": False,
         "factor": 1.0},
        # a prompt's query heads, normalised, the last third of each rotated
        {"name": "rope_prompt", "op": "rope", "n": 4096, "h": 128, "d": 192, "wide": 192, "out_wide": 192, "dims": 64, "norm": True, "interleaved": False,
         "factor": 4.0},
        # one row per sequence of a decoding step
        {"name": "place_bf16_step", "op": "place", "fp8": False, "d": 576, "n": 64, "pad": 0, "rows": False, "interleaved": True, "factor": 40.0},
        # a prompt of odd length with padding rows, kept as rows too for the up-projection
        {"name": "place_bf16_rows", "op": "place", "fp8": False, "d": 576, "n": 4999, "pad": 57, "rows": True, "interleaved": False, "factor": 1.0},
        # packed prompts into an e4m3 cache
        {"name": "place_fp8_prompt", "op": "place", "fp8": True, "d": 576, "n": 32768, "pad": 0, "rows": False, "interleaved": True, "factor": 40.0},
        # one short prompt with few heads: latency
        {"name": "prefill_short", "op": "prefill", "b": 1, "hq": 16, "hkv": 16, "rope": True, "lo": 333, "hi": 333, "ctx_lo": 0, "ctx_hi": 0, "causal": True, "pad": 0},
        # chunks of new tokens behind long contexts that were read back and up-projected: few rows, many keys
        {"name": "prefill_chunks", "op": "prefill", "b": 3, "hq": 16, "hkv": 16, "rope": True, "lo": 33, "hi": 256, "ctx_lo": 2000, "ctx_hi": 16384, "causal": True,
         "pad": 0},
        # packed prompts of many lengths, four query heads to a key head, no RoPE part
        {"name": "prefill_grouped", "op": "prefill", "b": 12, "hq": 32, "hkv": 8, "rope": False, "lo": 1, "hi": 2048, "ctx_lo": 0, "ctx_hi": 0, "causal": True, "pad": 65},
        # a whole prompt at all 128 heads: bound by the tensor cores
        {"name": "prefill_prompt", "op": "prefill", "b": 1, "hq": 128, "hkv": 128, "rope": True, "lo": 4096, "hi": 4096, "ctx_lo": 0, "ctx_hi": 0, "causal": True, "pad": 0},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "rope", "place", "place", "prefill", "prefill", "prefill"])
    if op == "pages":
        b = _spread(rng, 1, 1500)
        hi = _spread(rng, 1, min(8192, max(1, 131072 // b)))
        return {"op": op, "b": b, "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi, "past": rng.randint(0, 4096), "pad": rng.choice([0, 1, rng.randint(2, 100)]),
                "short": rng.random() < 0.4}
    factor = rng.choice([1.0, 4.0, 40.0])
    if op == "rope":
        h = rng.choice([1, 8, 16, 40, 128, rng.randint(1, 160)])
        norm = rng.random() < 0.6
        d, wide, out_wide, dims = rng.choice([(192, 192, 192, 64), (128, 128, 128, 128), (128, 256, 128, 32), (576, 576, 576, 64)] if norm else
                                             [(64, 192, 576, 64), (64, 64, 64, 64), (192, 192, 192, 64), (128, 128, 192, 128)])
        n = _spread(rng, 1, max(1, (4096 * 128 * 192) // (h * max(wide, out_wide))))
        return {"op": op, "n": n, "h": h, "d": d, "wide": wide, "out_wide": out_wide, "dims": dims, "norm": norm, "interleaved": rng.random() < 0.5, "factor": factor}
    if op == "place":
        fp8 = rng.random() < 0.5
        return {"op": op, "fp8": fp8, "d": 576 if fp8 or rng.random() < 0.75 else 512, "n": _spread(rng, 1, 32768), "pad": rng.choice([0, 0, 1, rng.randint(2, 100)]),
                "rows": rng.random() < 0.5, "interleaved": rng.random() < 0.5, "factor": factor}
    hkv = rng.choice([1, 2, 8, 16, 32])
    group = rng.choice([1, 1, 1, 2, 4, 5, 8, 16])
    if hkv == 32 and group == 1 and rng.random() < 0.5:
        hkv = 128
    hq = min(128, hkv * group) // hkv * hkv
    most = 128 * 4096 * 4096 // hq  # padded pairs of one head
    b = _spread(rng, 1, 32)
    hi = _spread(rng, 1, min(8192, int(math.sqrt(most // b))))
    span = min(16384, most // (b * hi) - hi)
    ctx_hi = rng.choice([0, 0, max(0, rng.randint(0, max(0, span)))])
    ctx_lo = rng.choice([0, ctx_hi, -(hi // 2)]) if ctx_hi == 0 or rng.random() < 0.3 else ctx_hi // 2
    return {"op": op, "b": b, "hq": hq, "hkv": hkv, "rope": rng.random() < 0.6, "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi, "ctx_lo": min(ctx_lo, ctx_hi),
            "ctx_hi": ctx_hi, "causal": rng.random() < 0.75, "pad": rng.choice([0, 0, 1, rng.randint(2, 200)])}


# ---------------------------------------------------------------- inputs
def _lengths(case):
    """Rows of each sequence (and keys, of a prefill): the case's own, so that buffers have one size."""
    g = torch.Generator().manual_seed(11 * case["b"] + case["hi"])
    count = torch.randint(case["lo"], case["hi"] + 1, (case["b"],), generator=g)
    count[-1] = case["hi"]  # the longest is always there
    if case["op"] != "prefill":
        return count, None
    ctx = torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (case["b"],), generator=g)
    return count, (count + ctx).clamp(min=0)


def _cu(count):
    return torch.nn.functional.pad(count.cumsum(0), (1, 0))


def _frequencies(dims, factor):
    """Radians per position of each pair: base 10000, of which the slow ones are stretched by ``factor`` for contexts
    longer than 4096 positions (a ramp between 32 turns in the 4096 and 1 turn)."""
    f = [10000.0 ** (-2.0 * i / dims) for i in range(dims // 2)]
    if factor == 1.0:
        return f
    pair = [dims * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32.0, 1.0)]
    lo, hi = max(0, math.floor(pair[0])), min(dims - 1, math.ceil(pair[1]))
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(dims // 2)]
    return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)]


def _turns(freq):
    """The same as the library takes them: turns per position in units of 2^-64."""
    units = [round(x / (2 * math.pi) * 2.0 ** 64) for x in freq]
    return torch.tensor([u - (1 << 64) if u >= 1 << 63 else u for u in units], dtype=torch.int64)


def _cache(g, nblk, d, fp8, dev):
    """A pool with something in every page."""
    if fp8:
        pages = torch.randint(0, 0x70, (nblk, PAGE * (d + 4)), generator=g, device=dev, dtype=torch.uint8)
        pages[:, PAGE * d:] = torch.full((nblk, PAGE), 0.01, device=dev).view(torch.uint8)
        return pages
    return torch.randn((nblk, PAGE, 1, d), generator=g, device=dev).to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    gc = torch.Generator()
    gc.manual_seed(seed)
    op = case["op"]
    state = {"case": case, "op": op, "dev": dev}
    to = lambda t, kind=torch.int32: t.to(kind).to(dev)  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    if op == "pages":
        b = case["b"]
        count, _ = _lengths(case)
        past = torch.randint(0, case["past"] + 1, (b,), generator=gc)
        have, width = (past + PAGE - 1) // PAGE, (case["past"] + case["hi"] + PAGE - 1) // PAGE + 1
        new = int(((past + count + PAGE - 1) // PAGE - have).sum())
        free = min(b * width, new * 2 // 3 if case["short"] else new + 5)
        pool = torch.randperm(2 * b * width, generator=gc)  # the table's pages are taken from its front, the free ones are its back half
        used = torch.arange(width)[None] < have[:, None]
        table = torch.full((b, width), -1, dtype=torch.int64)
        table[used] = pool[:int(have.sum())]
        n = int(count.sum()) + case["pad"]
        state |= {"lens": to(past), "cu": to(_cu(count)), "n": n, "table": to(table),
                  "free": to(pool[b * width:]), "left": to(torch.tensor([free]))}
        state |= {"left_out": torch.zeros_like(state["left"]), "lens_out": torch.zeros_like(state["lens"]),
                  "pos": torch.zeros((n,), dtype=torch.int32, device=dev), "slots": torch.zeros((n,), dtype=torch.int64, device=dev)}
        return state
    if op in ("rope", "place"):
        dims = case["dims"] if op == "rope" else ROPE
        freq = _frequencies(dims, case["factor"])
        far = 4096 * case["factor"]
        state |= {"freq": torch.tensor(freq, dtype=torch.float64, device=dev), "turns": _turns(freq).to(dev), "interleaved": case["interleaved"],
                  "mscale": 0.1 * math.log(case["factor"]) + 1.0}
    if op == "rope":
        n, h, d, dims = case["n"], case["h"], case["d"], case["dims"]
        state |= {"pos": to(torch.randint(0, int(far), (n,), generator=gc)), "dims": dims,
                  "x": (1.5 * randn(n, h, case["wide"])).to(torch.bfloat16)[..., case["wide"] - d:],
                  "out": torch.zeros((n, h, case["out_wide"]), dtype=torch.bfloat16, device=dev)[..., case["out_wide"] - d:],
                  "weight": (1.0 + 0.3 * randn(d)).to(torch.bfloat16) if case["norm"] else None}
        return state
    if op == "place":
        d, n, total = case["d"], case["n"], case["n"] + case["pad"]
        nblk = n // PAGE + 9
        both = (0.7 * randn(total, d)).to(torch.bfloat16)  # one projection's output
        slots = torch.full((total,), -1, dtype=torch.int64)
        slots[:n] = (torch.randperm(nblk, generator=gc)[:, None] * PAGE + torch.arange(PAGE)).view(-1)[3:3 + n]  # runs of rows, the first begun inside a page
        rows = torch.zeros((total, d), dtype=torch.bfloat16, device=dev) if case["rows"] else None
        state |= {"fp8": case["fp8"], "d": d, "n": total, "pos": to(torch.randint(0, int(far), (1,), generator=gc) + torch.arange(total)),
                  "latent": both[:, :LATENT], "rope": both[:, LATENT:] if d > LATENT else None, "slots": slots.to(dev),
                  "weight": (1.0 + 0.3 * randn(LATENT)).to(torch.bfloat16), "cache": _cache(g, nblk, d, case["fp8"], dev),
                  "latent_out": rows[:, :LATENT] if case["rows"] else None, "rope_out": rows[:, LATENT:] if case["rows"] and d > LATENT else None}
        return state
    lq, lk = _lengths(case)
    nq, nk = int(lq.sum()) + case["pad"], int(lk.sum()) + case["pad"]
    hq, hkv = case["hq"], case["hkv"]
    dq = HEAD + (ROPE if case["rope"] else 0)
    up = randn(max(1, nk), hkv, 2 * HEAD).to(torch.bfloat16)  # keys and values of one up-projection
    state |= {"cu_q": to(_cu(lq)), "cu_k": to(_cu(lk)), "most_q": case["hi"], "most_k": int(lk.max()), "nq": nq, "nk": nk, "scale": dq ** -0.5,
              "q": (2.0 * randn(max(1, nq), hq, dq)).to(torch.bfloat16), "k": up[..., :HEAD], "v": up[..., HEAD:],
              "k_rope": randn(max(1, nk), ROPE).to(torch.bfloat16) if case["rope"] else None,
              "out": torch.zeros((max(1, nq), hq, HEAD), dtype=torch.bfloat16, device=dev), "lse": torch.zeros((max(1, nq), hq), device=dev)}
    return state


# ---------------------------------------------------------------- plain forms
def _rows_of(cu, n, dev):
    """For every row: (is it of a sequence, its sequence, its place in it)."""
    r = torch.arange(n, device=dev)
    seq = torch.bucketize(r, cu[1:].long(), right=True)
    live = seq < cu.numel() - 1
    seq = seq.clamp(max=cu.numel() - 2)
    return live, seq, r - cu.long()[seq]


def _pages(state):
    lens, cu, table, left, dev = state["lens"].long(), state["cu"].long(), state["table"], state["left"].long(), state["dev"]
    new = lens + cu[1:] - cu[:-1]
    have = (lens + PAGE - 1) // PAGE
    need = (new + PAGE - 1) // PAGE - have
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= left)
    col = torch.arange(table.shape[1], device=dev)
    k = (upto - need - have)[:, None] + col  # which page of the list
    fresh = served[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    page = state["free"][(left - 1 - k).clamp(0, state["free"].numel() - 1)]
    table.copy_(torch.where(fresh, page, table))
    state["lens_out"].copy_(torch.where(served, new, lens))
    state["left_out"].copy_(left - torch.where(served, need, 0).sum())
    live, seq, i = _rows_of(cu, state["n"], dev)
    live = live & served[seq]
    pos = torch.where(live, lens[seq] + i, 0)
    state["pos"].copy_(pos)
    state["slots"].copy_(torch.where(live, table[seq, pos // PAGE].long() * PAGE + pos % PAGE, -1))
    return [table, state["lens_out"], state["left_out"], state["pos"], state["slots"]]


def _norm(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _rotate(state, x, dims):
    """fp32 x [n, h, d] with the last ``dims`` of d rotated."""
    angle = state["pos"].double()[:, None] * state["freq"]
    c, s = [(f(angle) * state["mscale"]).float()[:, None] for f in (torch.cos, torch.sin)]
    keep, x = x[..., :-dims], x[..., -dims:]
    if state["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.cat([keep, torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)], -1)
    a, b = x[..., :dims // 2], x[..., dims // 2:]
    return torch.cat([keep, a * c - b * s, b * c + a * s], -1)


def _rope(state):
    state["out"].copy_(_rotate(state, _norm(state["x"], state["weight"]), state["dims"]))
    return state["out"]


def _codes(state):
    """The pages' codes [n, 64, d] and scales [n, 64], as views."""
    d, pages = state["d"], state["cache"]
    return (pages[:, :PAGE * d].view(torch.float8_e4m3fn).unflatten(1, (PAGE, d)),
            pages[:, PAGE * d:].view(torch.float32))


def _placed(state):
    """What a pass over the rows leaves behind."""
    out = list(_codes(state)) if state["fp8"] else [state["cache"]]
    return out + [t for t in (state["latent_out"], state["rope_out"]) if t is not None]


def _place(state):
    x = _norm(state["latent"], state["weight"])
    if state["rope"] is not None:
        x = torch.cat([x, _rotate(state, state["rope"].float()[:, None], ROPE)[:, 0]], 1)
    if state["latent_out"] is not None:
        state["latent_out"].copy_(x[:, :LATENT])
    if state["rope_out"] is not None:
        state["rope_out"].copy_(x[:, LATENT:])
    live = state["slots"] >= 0
    blk, off, x = state["slots"][live] // PAGE, state["slots"][live] % PAGE, x[live]
    if state["fp8"]:
        amax = x.abs().amax(1)
        scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), 1.0)
        codes, scales = _codes(state)
        codes.view(torch.uint8)[blk, off] = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[blk, off] = scale
    else:
        state["cache"][blk, off, 0] = x.bfloat16()
    return _placed(state)


def _prefill(state):
    case, dev = state["case"], state["dev"]
    cu_q, cu_k = state["cu_q"].long(), state["cu_k"].long()
    b, hq, hkv, mq, mk = case["b"], case["hq"], case["hkv"], state["most_q"], max(1, state["most_k"])
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(mq, device=dev), torch.arange(mk, device=dev)
    at_q = (cu_q[:-1, None] + i).clamp(max=state["q"].shape[0] - 1)  # padded to the longest
    at_k = (cu_k[:-1, None] + j).clamp(max=state["k"].shape[0] - 1)
    there_q, there_k = i < lq[:, None], j < lk[:, None]
    q = state["q"][at_q].float().permute(0, 2, 1, 3).reshape(b, hkv, hq // hkv * mq, -1)  # [b, hkv, group and row, d]
    k = torch.where(there_k[..., None, None], state["k"][at_k], 0.0).float().permute(0, 2, 1, 3)
    v = torch.where(there_k[..., None, None], state["v"][at_k], 0.0).float().permute(0, 2, 1, 3)
    if state["k_rope"] is not None:
        k = torch.cat([k, torch.where(there_k[..., None], state["k_rope"][at_k], 0.0).float()[:, None].expand(b, hkv, mk, ROPE)], -1)
    seen = there_k[:, None, :].expand(b, mq, mk)
    if case["causal"]:
        seen = seen & (j < (lk - lq)[:, None, None] + i[:, None] + 1)
    z = (torch.matmul(q, k.transpose(-1, -2)) * state["scale"]).view(b, hkv, hq // hkv, mq, mk)
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, -1, mk), v).view(b, hq, mq, HEAD) / torch.where(total > 0, total, 1.0).view(b, hq, mq, 1)
    lse = (torch.log(total) + top).view(b, hq, mq)
    rows = at_q[there_q]
    state["out"][rows] = o.permute(0, 2, 1, 3)[there_q].bfloat16()
    state["lse"][rows] = lse.permute(0, 2, 1)[there_q]
    return [state["out"], state["lse"]]


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if own:
        import mla_decode_attention_latent_gb300 as mla
        if op == "pages":
            mla.mla_assign_pages(state["lens"], state["cu"], state["table"], state["free"], state["left"], state["n"], num_free_out=state["left_out"],
                                 new_seqlens=state["lens_out"], positions=state["pos"], slots=state["slots"])
            return [state["table"], state["lens_out"], state["left_out"], state["pos"], state["slots"]]
        if op == "rope":
            return mla.mla_norm_rope(state["x"], state["pos"], state["turns"], weight=state["weight"], eps=EPS, interleaved=state["interleaved"],
                                     rope_scale=state["mscale"], out=state["out"])
        if op == "place":
            place = mla.mla_norm_rope_cache_write_fp8 if state["fp8"] else mla.mla_norm_rope_cache_write
            roped = state["rope"] is not None
            place(state["latent"], state["rope"], state["pos"] if roped else None, state["turns"] if roped else None, state["slots"], state["cache"],
                  weight=state["weight"], eps=EPS, interleaved=state["interleaved"], rope_scale=state["mscale"], latent_out=state["latent_out"],
                  k_rope_out=state["rope_out"])
            return _placed(state)
        return list(mla.mla_prefill(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"], k_rope=state["k_rope"], softmax_scale=state["scale"],
                                    causal=state["case"]["causal"], out=state["out"], lse=state["lse"]))
    return {"pages": _pages, "rope": _rope, "place": _place, "prefill": _prefill}[op](state)


def work(case):
    op = case["op"]
    if op == "pages":
        n = float(_lengths(case)[0].sum()) + case["pad"]
        return {"bytes": 12.0 * n + case["b"] * 12.0 + n / PAGE * 8.0, "flops": 0.0}
    if op == "rope":
        values = float(case["n"] * case["h"] * case["d"])
        return {"bytes": 4.0 * values + 4.0 * case["n"], "flops": 4.0 * values if case["norm"] else 3.0 * values}
    if op == "place":
        d, n, total = case["d"], case["n"], case["n"] + case["pad"]
        row = d + 4 if case["fp8"] else 2 * d
        return {"bytes": float((total if case["rows"] else n) * 2 * d + n * row + (total * 2 * d if case["rows"] else 0) + total * 12), "flops": 5.0 * total * d}
    lq, lk = _lengths(case)
    dq = HEAD + (ROPE if case["rope"] else 0)
    if case["causal"]:  # row i sees keys up to lk - lq + i
        last, first = lk, (lk - lq + 1)
        low = first.clamp(min=1)
        pairs = float(((low + last) * (last - low + 1).clamp(min=0) // 2).sum())
    else:
        pairs = float((lq * lk).sum())
    nq, nk = float(lq.sum()), float(lk.sum())
    return {"bytes": nq * case["hq"] * (2 * dq + 2 * HEAD + 4) + nk * (case["hkv"] * 4 * HEAD + 2 * (dq - HEAD)), "flops": 2.0 * (dq + HEAD) * case["hq"] * pairs}


# ---------------------------------------------------------------- in 64 bits
def _exact_norm(x, weight):
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()


def _exact_turn(state, x, dims):
    """The last ``dims`` of x [n, h, d] as complex numbers, turned."""
    x = x.clone()
    part = x[..., x.shape[-1] - dims:]
    half = dims // 2
    re, im = (part[..., 0::2], part[..., 1::2]) if state["interleaved"] else (part[..., :half], part[..., half:])
    angle = torch.outer(state["pos"].double(), state["freq"])
    z = torch.complex(re, im) * torch.polar(torch.full_like(angle, state["mscale"]), angle)[:, None]
    re.copy_(z.real)
    im.copy_(z.imag)
    return x


def _exact_pages(state):
    lens, cu, table, free = [state[k].tolist() for k in ("lens", "cu", "table", "free")]
    left, asked = state["left"].tolist()[0], 0
    taken, after = 0, []
    pos, slots = [0] * state["n"], [-1] * state["n"]
    for b, old in enumerate(lens):
        new = old + cu[b + 1] - cu[b]
        need = -(-new // PAGE) - -(-old // PAGE)
        asked += need
        if need and asked > left:
            after.append(old)
            continue
        for c in range(-(-old // PAGE), -(-new // PAGE)):
            table[b][c] = free[left - 1 - taken]
            taken += 1
        after.append(new)
        for p in range(old, new):
            r = cu[b] + p - old
            pos[r], slots[r] = p, table[b][p // PAGE] * PAGE + p % PAGE
    make = lambda x, like: torch.tensor(x, dtype=like.dtype, device=like.device).view(like.shape)  # noqa: E731
    return [make(table, state["table"]), make(after, state["lens"]), make([left - taken], state["left"]), make(pos, state["pos"]), make(slots, state["slots"])]


def exact(case, seed):
    state = prepare(case, seed)
    op = state["op"]
    if op == "pages":
        return _exact_pages(state)
    if op == "rope":
        x = state["x"].double()
        return _exact_turn(state, x if state["weight"] is None else _exact_norm(x, state["weight"]), state["dims"])
    if op == "place":
        x = _exact_norm(state["latent"].double(), state["weight"])
        rows = [x]
        if state["rope"] is not None:
            rows.append(_exact_turn(state, state["rope"].double()[:, None], ROPE)[:, 0])
        x = torch.cat(rows, 1)
        slots = state["slots"]
        at = slots[slots >= 0]
        x = x[slots >= 0]
        if state["fp8"]:
            codes, scales = [t.double() for t in _codes(state)]
            big = x.abs().max(1).values
            c = torch.where(big > 0, big / 448, torch.ones_like(big))
            codes.view(-1, state["d"])[at] = (x / c[:, None]).float().to(torch.float8_e4m3fn).double()
            scales.view(-1)[at] = c
            out = [codes, scales]
        else:
            out = [state["cache"].double()]
            out[0].view(-1, state["d"])[at] = x
        return out + (rows if case["rows"] else [])
    hq, hkv = case["hq"], case["hkv"]
    cu_q, cu_k = state["cu_q"].tolist(), state["cu_k"].tolist()
    o, lse = torch.zeros(state["out"].shape, dtype=torch.float64, device=state["dev"]), torch.zeros(state["lse"].shape, dtype=torch.float64, device=state["dev"])
    for b in range(case["b"]):
        q = state["q"][cu_q[b]:cu_q[b + 1]].double()
        k, v = state["k"][cu_k[b]:cu_k[b + 1]].double(), state["v"][cu_k[b]:cu_k[b + 1]].double()
        if not q.shape[0]:
            continue
        behind = k.shape[0] - q.shape[0]
        hidden = torch.ones((q.shape[0], k.shape[0]), dtype=torch.bool, device=state["dev"]).triu(behind + 1) if case["causal"] else None
        for h in range(hq):
            y = q[:, h, :HEAD] @ k[:, h // (hq // hkv)].T
            if state["k_rope"] is not None:
                y += q[:, h, HEAD:] @ state["k_rope"][cu_k[b]:cu_k[b + 1]].double().T
            y *= state["scale"]
            if hidden is not None:
                y.masked_fill_(hidden, -math.inf)
            if not k.shape[0]:
                lse[cu_q[b]:cu_q[b + 1], h] = -math.inf
                continue
            each = torch.logsumexp(y, 1)
            lse[cu_q[b]:cu_q[b + 1], h] = each
            o[cu_q[b]:cu_q[b + 1], h] = torch.exp(y - torch.where(each > -math.inf, each, 0.0)[:, None]) @ v[:, h // (hq // hkv)]
    return [o, lse]
