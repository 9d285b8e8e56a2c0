"""Plain 64-bit restatements of the cache, page-selection and draft-tree calls, for the tests.

Everything runs on the CPU, one row or page at a time; roundings appear only where the calls' definitions
(``include/mla_decode.h``) put them, as an explicit conversion to fp32.
"""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE, DV = 64, 512


def f32(x):
    return x.to(torch.float32).to(torch.float64)


def cache_rows(cache: torch.Tensor) -> torch.Tensor:
    """Rows [num_blocks, 64, d] of a cache, fp64 (e4m3: the exact scale * code)."""
    c = cache.cpu()
    if c.dtype == torch.bfloat16:
        return c[:, :, 0].double()
    d = c.shape[1] // PAGE - 4
    codes = c[:, :PAGE * d].contiguous().view(torch.float8_e4m3fn).view(-1, PAGE, d)
    scales = c[:, PAGE * d:].contiguous().view(torch.float32)
    return codes.double() * scales.double()[..., None]


def quantised_row(x: torch.Tensor):
    """(codes uint8 [d], scale fp32) of one row of bf16 values."""
    amax = x.float().abs().max()
    c = amax / torch.tensor(448.0) if amax > 0 else torch.tensor(1.0)
    code = (x.float() / c).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(x == 0, torch.zeros_like(code), code), c  # a zero's code is +0


def page_key(rows: torch.Tensor):
    """(int8 key, scale) of one page from its n present rows, fp64 [n, d]."""
    n, d = rows.shape
    x = torch.zeros((PAGE, d), dtype=torch.float64)
    x[:n] = f32(rows)
    while x.shape[0] > 1:
        x = f32(x[0::2] + x[1::2])
    mean = f32(x[0] / n)
    amax = mean.abs().max()
    if not torch.isfinite(mean).all():
        return torch.zeros((d,), dtype=torch.int8), float("nan")
    scale = f32(amax / 127) if amax > 0 else torch.tensor(1.0, dtype=torch.float64)
    return torch.round(f32(mean / scale)).to(torch.int8), float(scale)


def token_len(T: int, s_q: int, i: int, causal: bool) -> int:
    return max(0, T - s_q + i + 1 if causal else T)


def page_scores(q: torch.Tensor, keys: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """Scores of pages (keys [n, d] int8, scales [n]) for one query token q [h, d]."""
    q = q.double()
    amax = q.abs().amax(1, keepdim=True)
    unit = f32(torch.where(amax > 0, amax / 127, torch.ones_like(amax)))
    whole = torch.round(f32(q / unit))
    each = f32(unit * (whole @ keys.double().T))
    if not torch.isfinite(q).all():
        return torch.full((keys.shape[0],), float("nan"), dtype=torch.float64)
    return f32(each.amax(0) * scales.double())


def select(score, n: int, topk: int, sink: int, local: int):
    """Selected pages of n, ascending."""
    if n <= topk:
        return list(range(n))
    s = [math.inf if math.isnan(v) else v for v in score.tolist()]
    nan = [math.isnan(v) for v in score.tolist()]
    mid = sorted(range(sink, n - local), key=lambda p: (not nan[p], -s[p], p))[:topk - sink - local]
    return sorted(list(range(sink)) + mid + list(range(n - local, n)))


def attend(q: torch.Tensor, rows: torch.Tensor, scale: float, fp8: bool = False):
    """(o [h, 512], lse [h], a [h, 512]) of q [h, d] over rows [t, d]; a = sum of weight * |value|, for an e4m3
    cache with the further term of assert_attention."""
    h = q.shape[0]
    if rows.shape[0] == 0:
        return torch.zeros((h, DV), dtype=torch.float64), torch.full((h,), -math.inf, dtype=torch.float64), \
            torch.zeros((h, DV), dtype=torch.float64)
    z = q.double() @ rows.T * scale
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    a = p @ rows[:, :DV].abs()
    if fp8:
        c = rows.abs().amax(1) / 448  # the row's scale (1 for a row of zeros, whose values are 0)
        c = torch.where(c > 0, c, torch.ones_like(c))
        a = a + (p * c).amax(1, keepdim=True) / 8 * (rows[:, :DV].abs() / c[:, None]).sum(0)
    return p @ rows[:, :DV], lse, a


def assert_attention(o, lse, o_ref, lse_ref, a_ref, fp8: bool, what=""):
    """o and lse against 64 bits.

    Rounding o to bf16 is off by at most 2^-8 |o|.  The weights are rounded to bf16 (2^-8 each), and a score's
    fp32 accumulation adds less than 2^-11 of its weight, so the sum over the values is off by at most
    (2^-8 + 2^-11) * a, a = sum of weight * |value|.  e4m3: a weight times its token's scale, w_j = p_j c_j, is held
    in two e4m3 parts, each off by half a step: 2^-4 * 2^-4 of w_j, or half the smallest step, 2^-10, where the
    largest weight of the segment's first page is at least 3.5; 2^-10 / 3.5 < 2^-11 of the largest w, which adds
    2^-11 max w * sum |code| = 2^-8 * (max w / 8) * sum |value| / c to the bound: the term that attend adds to a.
    LSE: 2e-3, the library's bound for both caches."""
    o, lse = o.double().cpu(), lse.double().cpu()
    inf = torch.isneginf(lse_ref)
    assert torch.equal(torch.isneginf(lse), inf), f"{what}: pattern of empty rows"
    d = (lse - lse_ref)[~inf].abs()
    assert d.numel() == 0 or float(d.max()) <= 2e-3, f"{what}: |dLSE| = {float(d.max()):.3e}"
    assert torch.isfinite(o).all(), f"{what}: o is not finite"
    bound = 2.0 ** -8 * o_ref.abs() + (2.0 ** -8 + 2.0 ** -11) * a_ref + 1e-30
    worst = ((o - o_ref).abs() / bound).max()
    assert float(worst) <= 1.0, f"{what}: |dO| is {float(worst):.3f} times its bound"


def place(table, b: int, pos: int):
    return int(table[b, pos // PAGE]), pos % PAGE


def ancestors(parents) -> np.ndarray:
    """sees [s, s] of one tree."""
    s = len(parents)
    sees = np.zeros((s, s), bool)
    for i in range(s):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = parents[j]
    return sees


def mask_words(sees: np.ndarray) -> torch.Tensor:
    """int32 [s, ceil(s / 32)] of sees [s, s]."""
    s = sees.shape[0]
    out = np.zeros((s, (s + 31) // 32), np.uint32)
    for i in range(s):
        for j in range(s):
            if sees[i, j]:
                out[i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    return torch.from_numpy(out.view(np.int32).copy())


def random_cache(gen, nblk: int, d: int, fp8: bool):
    """A pool of N(0, 1) rows (CPU): bf16 [nblk, 64, 1, d] or packed e4m3 pages."""
    from mla_decode_attention_latent_gb300 import workloads as W
    x = torch.randn((nblk, PAGE, d), generator=gen)
    return W.pack_e4m3_pages(x) if fp8 else x[:, :, None].to(torch.bfloat16)


def random_table(gen, lens, nblk=None, extra=0):
    """(table int32 [b, width], pages used) with distinct pages per sequence."""
    need = [(t + PAGE - 1) // PAGE for t in lens]
    width = max(1, max(need)) + extra
    nblk = max(1, sum(need)) if nblk is None else nblk
    perm = torch.randperm(nblk, generator=gen).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, nblk
