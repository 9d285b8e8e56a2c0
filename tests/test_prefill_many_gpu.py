"""Prompt attention over hundreds of sequences of which some are cut: the partition of a thousand threads, with and without cuts."""
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from tests.test_prefill_gpu import check, cu_of, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.mark.parametrize("b,hq,hkv,longest", [(300, 2, 1, [20000, 5000, 12345]), (300, 2, 2, [16384, 9000]), (300, 4, 1, []), (700, 1, 1, [8000] * 6),
                                              (1000, 2, 1, [20000, 7000, 5000, 15000])])
@pytest.mark.parametrize("causal", [True, False])
def test_hundreds_of_sequences(dev, b, hq, hkv, longest, causal):
    """More sequences or blocks than 256, contexts of all lengths, no more blocks than the partition keeps at once."""
    mla.mla_device_status()
    g = torch.Generator().manual_seed(b + hkv)
    lq = torch.randint(0, 4, (b,), generator=g).tolist()
    lk = [n + int(x) for n, x in zip(lq, torch.randint(0, 400, (b,), generator=g))]
    for at, n in zip(torch.randperm(b, generator=g).tolist(), longest):
        lq[at], lk[at] = max(1, lq[at]), n
    q, k, v, kr = make(dev, lq, lk, hq, hkv, False, seed=b)
    cq, ck = cu_of(lq, dev), cu_of(lk, dev)
    md = mla.mla_get_metadata_prefill(cq, ck, q.shape[0], k.shape[0], hq, hkv, causal=causal)
    segments, cuts = md[:2].tolist()
    live = sum(1 for n in lq if n)
    assert (cuts > 0 and segments > live) if longest else (cuts == 0 and segments == live)
    out, lse = mla.mla_prefill(q, k, v, cq, ck, causal=causal, metadata=md)
    check(out, lse, q, k, v, kr, lq, lk, causal)
    again, lse2 = mla.mla_prefill(q, k, v, cq, ck, causal=causal)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert mla.mla_device_status() == 0
