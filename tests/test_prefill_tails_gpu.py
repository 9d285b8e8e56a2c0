"""Prompt attention where a warp's rows are partly of no query: sequences that end at every lane, whole blocks and cut ones."""
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from tests.test_prefill_gpu import check, cu_of, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.mark.parametrize("group", [1, 3, 5])
@pytest.mark.parametrize("context", [0, 3000])
@pytest.mark.parametrize("rope", [True, False])
def test_sequences_that_end_at_every_lane(dev, group, context, rope):
    mla.mla_device_status()
    tokens = 128 // group
    # rows that end at each lane of a tile's first and last warps, and of the second tile's
    lq = [n for n in range(1, 2 * tokens + 2) if n * group % 128 < 36 or n * group % 128 > 92]
    lq = lq[::1 if context == 0 else 9]
    lk = [n + (context if i % 3 == 0 else 0) for i, n in enumerate(lq)]
    q, k, v, kr = make(dev, lq, lk, group, 1, rope, seed=group, pad=7)
    cq, ck = cu_of(lq, dev), cu_of(lk, dev)
    n = sum(lq)
    out, lse = torch.full((n + 7, group, 128), 5.0, dtype=torch.bfloat16, device=dev), torch.full((n + 7, group), 5.0, device=dev)
    md = mla.mla_get_metadata_prefill(cq, ck, n + 7, k.shape[0], group, 1)
    if context:
        assert md[1].item() > 0  # some are cut
    mla.mla_prefill(q, k, v, cq, ck, k_rope=kr, out=out, lse=lse, metadata=md)
    check(out, lse, q, k, v, kr, lq, lk, True)
    assert (out[n:] == 5).all() and (lse[n:] == 5).all()
    assert mla.mla_device_status() == 0
