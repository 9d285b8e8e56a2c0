"""Page keys of means so small that their scale is subnormal."""
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import workloads as W
from tests import reference64 as R

pytestmark = pytest.mark.gpu


def page_key(rows):
    """R.page_key with the limits of a subnormal scale: at least 2^-149, keys at most 127."""
    x = torch.zeros((64, rows.shape[1]), dtype=torch.float64)
    x[:rows.shape[0]] = R.f32(rows)
    while x.shape[0] > 1:
        x = R.f32(x[0::2] + x[1::2])
    mean = R.f32(x[0] / rows.shape[0])
    amax = float(mean.abs().max())
    scale = max(float(R.f32(torch.tensor(amax, dtype=torch.float64) / 127)), 2.0 ** -149) if amax else 1.0
    return torch.round(R.f32(mean / scale)).clamp(-127, 127).to(torch.int8), scale


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 5, 64, 64 + 33])
def test_page_keys_of_the_smallest_rows(fp8, n):
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(n)
    mla.mla_device_status()
    pages = (n + 63) // 64
    for size in range(14):
        # bf16's own subnormals are multiples of 2^-133; e4m3 pages reach every fp32 one through their scales
        rows = torch.zeros((pages, 64, 576))
        rows[:, size % 3, ::(7 if size % 2 else 1)] = 1.0
        rows[:, 0] += torch.randint(-1, 2, (576,), generator=g)
        if fp8:
            cache = W.pack_e4m3_pages(rows, torch.full((pages, 64), 2.0 ** -149 * (1 << size)))
        else:
            cache = (rows * 2.0 ** -133 * (1 + size // 2)).to(torch.bfloat16)[:, :, None]
        assert R.cache_rows(cache).abs().max() > 0
        table = torch.arange(pages, dtype=torch.int32)[None]
        keys = torch.full((pages, 576), 99, dtype=torch.int8, device=dev)
        scales = torch.full((pages,), 99.0, device=dev)
        (mla.mla_update_page_keys_fp8 if fp8 else mla.mla_update_page_keys)(
            cache.to(dev), table.to(dev), torch.tensor([n], dtype=torch.int32, device=dev), keys, scales)
        assert mla.mla_device_status() == 0
        for p in range(pages):
            k, s = page_key(R.cache_rows(cache)[p, :min(64, n - 64 * p)])
            assert torch.equal(keys[p].cpu(), k), (size, p)
            assert float(scales[p]) == s, (size, p)
