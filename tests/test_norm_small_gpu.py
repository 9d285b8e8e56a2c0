"""Norms of rows down to the smallest bf16 values, against the formula in 64 bits.

Bounds: those of test_norm_rope_gpu.  Where a row is scaled by a power of two first, that changes no digit of a value or
of a sum: nothing is added to them.
"""
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib
from tests import reference64 as R
from tests.test_norm_rope_gpu import formula, near

pytestmark = pytest.mark.gpu
PAGE = 64
SIZES = (0, 20, 44, 46, 60, 75, 100, 120, 126, 128, 130, 131, 132)  # a row's values are about 2^-size


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_status_left():
    mla.mla_device_status()
    yield


def tiny(shape, seed):
    """bf16 rows of every size side by side, a fifth of the values zero, no row of zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float64)
    x[torch.rand(shape, generator=g) < 0.2] = 0.0
    size = torch.tensor(SIZES, dtype=torch.float64)[torch.arange(shape[0] * shape[1]) % len(SIZES)].view(*shape[:2], 1)
    x = (x * torch.exp2(-size)).to(torch.bfloat16)
    x[..., 0] = torch.exp2(-size[..., 0]).to(torch.bfloat16)
    return x


@pytest.mark.parametrize("d,dims,h,n", [(64, 0, 3, 26), (64, 64, 2, 39), (128, 128, 5, 13), (192, 64, 3, 26), (200, 48, 2, 13), (256, 64, 1, 26), (576, 64, 2, 13),
                                        (320, 96, 1, 13)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -100, 2.0 ** -61, 2.0 ** -60, 1e-6])
def test_heads(dev, d, dims, h, n, interleaved, eps):
    x = tiny((n, h, d), d + n).to(dev)
    g = torch.Generator().manual_seed(d)
    w = (1 + 0.5 * torch.randn((d,), generator=g)).to(torch.bfloat16).to(dev)
    turns = mla.mla_rope_turns(dims, device=dev) if dims else None
    pos = torch.arange(n, dtype=torch.int32, device=dev) if dims else None
    eps = float(torch.tensor(eps, dtype=torch.float32))
    got = mla.mla_norm_rope(x, pos, turns, weight=w, eps=eps, interleaved=interleaved)
    near(got, *formula(x, pos, turns, w, eps, interleaved, 1.0))
    y = x.clone()
    mla.mla_norm_rope(y, pos, turns, weight=w, eps=eps, interleaved=interleaved, out=y)
    assert torch.equal(y, got)


@pytest.mark.parametrize("d", [576, 512])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -60])
def test_placed_rows(dev, d, eps):
    n = 2 * len(SIZES)
    both = torch.cat([tiny((n, 1, 512), d)[:, 0], tiny((1, 1, 64), 1)[0].expand(n, 64)], 1)[:, :d].contiguous().to(dev)
    g = torch.Generator().manual_seed(d)
    w = (1 + 0.5 * torch.randn((512,), generator=g)).to(torch.bfloat16).to(dev)
    rope = d > 512
    turns, pos = mla.mla_rope_turns(64, device=dev), torch.arange(n, dtype=torch.int32, device=dev)
    args = (both[:, :512], both[:, 512:] if rope else None, pos if rope else None, turns if rope else None, torch.arange(n, device=dev))
    want, bound = formula(both[:, None, :512], None, None, w, eps, False, 1.0)
    if rope:
        more = formula(both[:, None, 512:], pos, turns, None, 0, False, 1.0)
        want, bound = torch.cat([want, more[0]], -1), torch.cat([bound, more[1]], -1)
    want, bound = want[:, 0], bound[:, 0]
    cache = torch.zeros((1, PAGE, 1, d), dtype=torch.bfloat16, device=dev)
    out = torch.zeros((n, d), dtype=torch.bfloat16, device=dev)
    mla.mla_norm_rope_cache_write(*args, cache, weight=w, eps=eps, latent_out=out[:, :512], k_rope_out=out[:, 512:] if rope else None)
    near(out, want, bound)
    assert torch.equal(cache.view(PAGE, d)[:n], out)
    if rope:
        pages = torch.zeros((1, _lib.MLA_FP8_PAGE_BYTES(576)), dtype=torch.uint8, device=dev)
        mla.mla_norm_rope_cache_write_fp8(*args, pages, weight=w, eps=eps)
        got = R.cache_rows(pages).view(-1, 576)[:n]
        scale = pages.cpu()[0, PAGE * 576:].contiguous().view(torch.float32)[:n].double()[:, None]
        ok = (got - want).abs() <= 2 * bound + 2.0 ** -4 * want.abs() + 2.0 ** -10 * scale
        assert bool(ok.all())
    assert mla.mla_device_status() == 0
