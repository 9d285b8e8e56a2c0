"""Norms and rotations of heads, and of rows on their way into the cache, against the formulas in 64 bits.

Bounds.  The kernels work in fp32: a norm's sum of at most 576 squares is at most 75 roundings deep (2^-24 each, halved
by the root), a sine or cosine is off by less than 2^-22, a product or sum by 2^-24, so a value is off by less than
2^-18 (|a| + |b|) times the scale, its pair before the rotation being (a, b); 2^-17 is asked.  Then one rounding: half a
step, 2^-8 of a bf16 value (2^-134 below its normal range, whose steps are 2^-133), 2^-4 of an e4m3 code or 2^-10 of a unit where codes are subnormal.
"""
import math

import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib
from tests import reference64 as R

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_status_left():
    mla.mla_device_status()
    yield


def formula(x, positions, turns, weight, eps, interleaved, scale):
    """(values, bound before the last rounding), fp64 on the CPU, of x [n, h, d]."""
    x = x.detach().cpu().double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.cpu().double()
    y, bound = x.clone(), x.abs() * 2.0 ** -17
    if turns is not None:
        units, half = [t % (1 << 64) for t in turns.tolist()], turns.numel()
        part = [((p * u) % (1 << 64)) for p in positions.tolist() for u in units]  # whole turns dropped, in integers
        t = torch.tensor([2 * math.pi * (k - (1 << 64) if k >= 1 << 63 else k) / 2.0 ** 64 for k in part], dtype=torch.float64).view(-1, 1, half)
        lo = x.shape[-1] - 2 * half
        ia = lo + (2 * torch.arange(half) if interleaved else torch.arange(half))
        ib = ia + (1 if interleaved else half)
        a, b = x[..., ia], x[..., ib]
        y[..., ia] = (a * t.cos() - b * t.sin()) * scale
        y[..., ib] = (b * t.cos() + a * t.sin()) * scale
        bound[..., ia] = bound[..., ib] = (a.abs() + b.abs()) * scale * 2.0 ** -17
    return y, bound


def near(got, want, bound):
    got = got.detach().cpu().double()
    inside = bool(((got - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound) + 2.0 ** -134).all())
    assert inside


@pytest.mark.parametrize("dims,base,factor,original", [(64, 10000.0, 1.0, 0), (64, 10000.0, 4.0, 0), (64, 10000.0, 40.0, 4096), (128, 5e5, 8.0, 8192),
                                                       (32, 1e6, 1.0, 4096), (64, 1e4, 2.5, 100)])
def test_turns(dims, base, factor, original):
    got = mla.mla_rope_turns(dims, base, factor, original, device="cpu").tolist()
    for i, units in enumerate(got):
        f = base ** (-2.0 * i / dims)
        r = 1.0
        if original:
            pair = [dims * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (32.0, 1.0)]
            lo, hi = max(0, math.floor(pair[0])), min(dims - 1, math.ceil(pair[1]))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        f = f / factor * r + f * (1 - r)
        # rounded to a whole unit of 2^-64 turns: off by half of one, 2^-65 turns, beside the formula's own roundings
        assert abs(units / 2.0 ** 64 * 2 * math.pi - f) <= f * 2.0 ** -48 + 2 * math.pi * 2.0 ** -65


# (d, rotated, heads, tokens): every head a group of lanes takes, odd counts, a part that starts off a lane's first piece
@pytest.mark.parametrize("d,dims,h,n", [(64, 64, 128, 64), (192, 64, 3, 77), (192, 64, 128, 9), (128, 128, 40, 33), (128, 32, 1, 301), (576, 64, 16, 21),
                                        (72, 16, 5, 50), (200, 48, 7, 13), (256, 256, 2, 40), (320, 96, 3, 5), (8, 0, 3, 70), (16, 16, 1, 1), (512, 64, 1, 1)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads(dev, d, dims, h, n, norm, interleaved):
    g = torch.Generator().manual_seed(d + dims + n)
    x = (torch.randn((n, h, d), generator=g) * torch.exp(torch.randn((n, h, 1), generator=g))).to(torch.bfloat16).to(dev)
    w = (1 + 0.5 * torch.randn((d,), generator=g)).to(torch.bfloat16).to(dev) if norm else None
    turns = mla.mla_rope_turns(dims, 10000.0, 40.0, 4096, device=dev) if dims else None
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32).to(dev) if dims else None
    want, bound = formula(x, pos, turns, w, 1e-6, interleaved, 1.25)
    got = mla.mla_norm_rope(x, pos, turns, weight=w, interleaved=interleaved, rope_scale=1.25)
    near(got, want, bound)
    if not norm:  # the rest is copied
        assert torch.equal(got[..., :d - dims], x[..., :d - dims])
    # in place, the same values
    y = x.clone()
    assert mla.mla_norm_rope(y, pos, turns, weight=w, interleaved=interleaved, rope_scale=1.25, out=y) is y
    assert torch.equal(y, got)


def test_slices_of_wider_heads(dev):
    n, h = 50, 17
    wide = torch.randn((n, h, 192), device=dev).to(torch.bfloat16)
    to = torch.full((n, h, 576), 7.0, dtype=torch.bfloat16, device=dev)
    turns, pos = mla.mla_rope_turns(64, device=dev), torch.arange(n, dtype=torch.int32, device=dev)
    mla.mla_norm_rope(wide[..., 128:], pos, turns, out=to[..., 512:])
    want, bound = formula(wide[..., 128:], pos, turns, None, 0, False, 1.0)
    near(to[..., 512:], want, bound)
    assert (to[..., :512] == 7).all()
    # heads outside tokens, and one key head for all (its head stride means nothing)
    x = torch.randn((h, n, 64), device=dev).to(torch.bfloat16).transpose(0, 1)
    out = torch.empty((h, n, 64), dtype=torch.bfloat16, device=dev).transpose(0, 1)
    mla.mla_norm_rope(x, pos, turns, out=out, interleaved=True)
    near(out, *formula(x, pos, turns, None, 0, True, 1.0))
    one = wide[:, 0, :64][:, None]
    near(mla.mla_norm_rope(one, pos, turns), *formula(one, pos, turns, None, 0, False, 1.0))


def test_far_and_negative_positions(dev):
    turns = mla.mla_rope_turns(64, device=dev)
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 31) - 1, -(1 << 31), 123456789], dtype=torch.int32, device=dev)
    x = torch.randn((7, 4, 64), device=dev).to(torch.bfloat16)
    for interleaved in (False, True):
        near(mla.mla_norm_rope(x, pos, turns, interleaved=interleaved), *formula(x, pos, turns, None, 0, interleaved, 1.0))


def test_odd_heads_of_values(dev):
    """Heads of zeros, of the largest and smallest values, and heads that are not finite, each for itself."""
    x = torch.randn((6, 2, 128), device=dev).to(torch.bfloat16)
    x[0, 0], x[1, 0], x[2, 0] = 0.0, 3e18, 1e-30
    x[5, 0, 3] = 3.3e38
    x[3, 0, 5], x[4, 0, 7] = math.nan, math.inf
    w = torch.ones((128,), dtype=torch.bfloat16, device=dev)
    got = mla.mla_norm_rope(x, None, None, weight=w)
    good = [(i, j) for i in range(6) for j in range(2) if (i, j) not in ((3, 0), (4, 0))]
    want, bound = formula(x, None, None, w, 1e-6, False, 1.0)
    for i, j in good:
        near(got[i, j], want[i, j], bound[i, j])
    # without an eps small heads are as good as any
    x = x[:3, 1:] * torch.tensor([1.0, 1e-18, 1e-36], device=dev, dtype=torch.bfloat16).view(3, 1, 1)
    near(mla.mla_norm_rope(x, None, None, weight=w, eps=0.0), *formula(x, None, None, w, 0.0, False, 1.0))
    assert got[3, 0].isnan().all() and got[4, 0, 7].isnan() and (got[4, 0, :7] == 0).all()


def test_no_tokens(dev):
    turns = mla.mla_rope_turns(64, device=dev)
    assert mla.mla_norm_rope(torch.empty((0, 4, 64), dtype=torch.bfloat16, device=dev), torch.empty((0,), dtype=torch.int32, device=dev), turns).shape == (0, 4, 64)


# ---------------------------------------------------------------- rows into the cache
def rows(dev, n, d, seed=0, nblk=None, spread=True):
    g = torch.Generator().manual_seed(seed)
    nblk = nblk or n // 32 + 2
    both = torch.randn((n, d), generator=g)
    if spread:
        both = both * torch.exp(torch.randn((n, 1), generator=g))
    slots = torch.randperm(nblk * PAGE, generator=g)[:n]
    slots[torch.rand((n,), generator=g) < 0.15] = -1
    pos = torch.randint(0, 200000, (n,), generator=g, dtype=torch.int32)
    w = (1 + 0.5 * torch.randn((512,), generator=g)).to(torch.bfloat16)
    return both.to(torch.bfloat16).to(dev), slots.to(dev), pos.to(dev), w.to(dev), nblk


def by_formula(both, pos, turns, w, interleaved, scale, d):
    lat, lb = formula(both[:, None, :512], None, None, w, 1e-6, False, 1.0)
    if d == 512:
        return lat[:, 0], lb[:, 0]
    rope, rb = formula(both[:, None, 512:], pos, turns, None, 0, interleaved, scale)
    return torch.cat([lat, rope], -1)[:, 0], torch.cat([lb, rb], -1)[:, 0]


@pytest.mark.parametrize("d", [576, 512])
@pytest.mark.parametrize("n", [1, 7, 8, 64, 333])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_bf16(dev, d, n, norm, interleaved):
    both, slots, pos, w, nblk = rows(dev, n, d, n + d)
    turns = mla.mla_rope_turns(64, 1e4, 40.0, 4096, device=dev) if d > 512 else None
    cache = torch.full((nblk, PAGE, 1, d), 3.0, dtype=torch.bfloat16, device=dev)
    out = torch.full((n, d), 9.0, dtype=torch.bfloat16, device=dev)
    rope = d > 512
    mla.mla_norm_rope_cache_write(both[:, :512], both[:, 512:] if rope else None, pos if rope else None, turns, slots, cache,
                                  weight=w if norm else None, interleaved=interleaved, rope_scale=0.75, latent_out=out[:, :512],
                                  k_rope_out=out[:, 512:] if rope else None)
    want, bound = by_formula(both, pos, turns, w if norm else None, interleaved, 0.75, d)
    near(out, want, bound)
    expect = torch.full((nblk * PAGE, d), 3.0, dtype=torch.bfloat16, device=dev)
    live = slots >= 0
    expect[slots[live]] = out[live]
    assert torch.equal(cache.view(-1, d), expect)  # the same rows, and nothing else touched
    assert mla.mla_device_status() == 0


@pytest.mark.parametrize("n", [1, 9, 64, 333])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_fp8(dev, n, norm, interleaved):
    both, slots, pos, w, nblk = rows(dev, n, 576, n)
    if n > 8:
        both[3] = 0.0  # a row of zeros: scale 1, codes 0
    turns = mla.mla_rope_turns(64, 1e4, 40.0, 4096, device=dev)
    pages = torch.full((nblk, _lib.MLA_FP8_PAGE_BYTES(576)), 0x5a, dtype=torch.uint8, device=dev)
    mla.mla_norm_rope_cache_write_fp8(both[:, :512], both[:, 512:], pos, turns, slots, pages, weight=w if norm else None,
                                      interleaved=interleaved, rope_scale=0.75)
    want, bound = by_formula(both, pos, turns, w if norm else None, interleaved, 0.75, 576)
    live = (slots >= 0).cpu()
    at = slots.cpu()[live]
    got = R.cache_rows(pages).view(-1, 576)[at]
    scale = pages.cpu()[:, PAGE * 576:].contiguous().view(torch.float32).view(-1)[at].double()[:, None]
    want, bound = want[live], bound[live]
    top = want.abs().amax(1, keepdim=True)
    ideal = torch.where(top > 0, top / 448, 1.0)
    assert ((scale - ideal).abs() <= ideal * 2.0 ** -16).all()
    assert ((got - want).abs() <= 2 * bound + 2.0 ** -4 * want.abs() + 2.0 ** -10 * scale).all()
    # other rows of the pages are left as they were
    rest = torch.ones((nblk * PAGE,), dtype=torch.bool)
    rest[at] = False
    assert (pages.cpu()[:, :PAGE * 576].reshape(-1, 576)[rest] == 0x5a).all()
    assert (pages.cpu()[:, PAGE * 576:].reshape(-1, 4)[rest] == 0x5a).all()
    assert mla.mla_device_status() == 0


def test_without_norm_or_rotation_it_is_the_cache_write(dev):
    """At position 0 and without a weight, the pages are those of mla_cache_write, bit for bit."""
    n = 200
    both, _, _, _, _ = rows(dev, n, 576, 3)
    both[5], both[6, :3] = 0.0, torch.tensor([-0.0, 1e-38, -3e-39])
    zero = torch.zeros((n,), dtype=torch.int32, device=dev)
    turns = mla.mla_rope_turns(64, device=dev)
    table, starts = torch.arange(4, dtype=torch.int32, device=dev)[None].contiguous(), torch.zeros((1,), dtype=torch.int32, device=dev)
    for fp8 in (False, True):
        shape, kind = ((4, _lib.MLA_FP8_PAGE_BYTES(576)), torch.uint8) if fp8 else ((4, PAGE, 1, 576), torch.bfloat16)
        a, b = torch.zeros(shape, dtype=kind, device=dev), torch.zeros(shape, dtype=kind, device=dev)
        (mla.mla_cache_write_fp8 if fp8 else mla.mla_cache_write)(both[:, :512], both[:, 512:], a, table, starts)
        (mla.mla_norm_rope_cache_write_fp8 if fp8 else mla.mla_norm_rope_cache_write)(
            both[:, :512], both[:, 512:], zero, turns, torch.arange(n, device=dev), b)
        assert torch.equal(a.view(torch.uint8) if fp8 else a.float(), b.view(torch.uint8) if fp8 else b.float())


def test_slots_past_the_pool_and_rows_that_are_not_finite(dev):
    both, _, pos, w, _ = rows(dev, 4, 576, 1)
    turns = mla.mla_rope_turns(64, device=dev)
    cache = torch.full((2, PAGE, 1, 576), 3.0, dtype=torch.bfloat16, device=dev)
    slots = torch.tensor([127, 128, 1 << 40, -(1 << 50)], device=dev)
    mla.mla_norm_rope_cache_write(both[:, :512], both[:, 512:], pos, turns, slots, cache, weight=w)
    assert mla.mla_device_status() == _lib.MLA_DEVERR_BLOCK_ID
    assert (cache.view(128, 576)[:127] == 3).all() and not (cache.view(128, 576)[127] == 3).any()
    pages = torch.zeros((2, _lib.MLA_FP8_PAGE_BYTES(576)), dtype=torch.uint8, device=dev)
    for value in (math.nan, math.inf):
        bad = both.clone()
        bad[2, 570] = value
        mla.mla_norm_rope_cache_write_fp8(bad[:, :512], bad[:, 512:], pos, turns, torch.arange(4, device=dev), pages, weight=w)
        scales = pages[0, PAGE * 576:].view(torch.float32)
        assert scales[2].isnan() and scales[[0, 1, 3]].isfinite().all()
        assert mla.mla_device_status() == _lib.MLA_DEVERR_SCALE


def test_pages_beyond_32_bits(dev):
    """Slots whose byte offset passes 2^32, in both formats."""
    both, _, pos, w, _ = rows(dev, 3, 576, 2)
    turns = mla.mla_rope_turns(64, device=dev)
    nblk = 120000
    slots = torch.tensor([nblk * PAGE - 1, 0, (1 << 32) // 1152 + 5], device=dev)
    cache = torch.zeros((nblk, PAGE, 1, 576), dtype=torch.bfloat16, device=dev)
    out = torch.empty((3, 576), dtype=torch.bfloat16, device=dev)
    mla.mla_norm_rope_cache_write(both[:, :512], both[:, 512:], pos, turns, slots, cache, weight=w, latent_out=out[:, :512], k_rope_out=out[:, 512:])
    assert torch.equal(cache.view(-1, 576)[slots], out)
    del cache
    pages = torch.zeros((nblk, _lib.MLA_FP8_PAGE_BYTES(576)), dtype=torch.uint8, device=dev)
    few = torch.zeros((1, _lib.MLA_FP8_PAGE_BYTES(576)), dtype=torch.uint8, device=dev)
    mla.mla_norm_rope_cache_write_fp8(both[:, :512], both[:, 512:], pos, turns, slots, pages, weight=w)
    mla.mla_norm_rope_cache_write_fp8(both[:, :512], both[:, 512:], pos, turns, torch.arange(3, device=dev), few, weight=w)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(pages[s // PAGE, (s % PAGE) * 576:(s % PAGE + 1) * 576], few[0, i * 576:(i + 1) * 576])
    assert mla.mla_device_status() == 0


@pytest.mark.parametrize("d", [128, 136, 192, 256, 320])
@pytest.mark.parametrize("norm", [False, True])
def test_rotations_of_128_values(dev, d, norm):
    """Halves of 64 values: in a lane's own pieces where the head has whole ones before them, elsewhere not."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn((41, 5, d + 8), generator=g).to(torch.bfloat16).to(dev)[..., :d]
    w = (1 + 0.5 * torch.randn((d,), generator=g)).to(torch.bfloat16).to(dev) if norm else None
    turns = mla.mla_rope_turns(128, 5e5, 8.0, 8192, device=dev)
    pos = torch.randint(0, 1 << 20, (41,), generator=g, dtype=torch.int32).to(dev)
    got = mla.mla_norm_rope(x, pos, turns, weight=w, rope_scale=0.75)
    near(got, *formula(x, pos, turns, w, 1e-6, False, 0.75))
    if not norm:
        assert torch.equal(got[..., :d - 128], x[..., :d - 128])
    y = x.clone()
    mla.mla_norm_rope(y, pos, turns, weight=w, rope_scale=0.75, out=y)
    assert torch.equal(y, got)
