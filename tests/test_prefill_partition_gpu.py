"""A prompt attention's partition used by a call of other shapes, with the same bounds: joined, or reported and nothing written."""
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib
from tests.test_prefill_gpu import check, cu_of, make

pytestmark = pytest.mark.gpu
CUTS = 1  # word of the partition: cut blocks


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_status_left():
    mla.mla_device_status()
    yield


def unset(q):
    return torch.full((*q.shape[:2], 128), 5.0, dtype=torch.bfloat16, device=q.device), torch.full(q.shape[:2], 5.0, device=q.device)


def test_cuts_that_a_call_of_more_rows_would_not_join(dev):
    """Made for 256 query rows over many keys, used with the rows padded: a call of so many rows enqueues no combine."""
    lq, lk, h = [256], [9000], 16
    pad = 8 * torch.cuda.get_device_properties(dev).multi_processor_count // h * 256  # blocks of the padded call: more than 8 items to a CTA
    q, k, v, kr = make(dev, lq, lk, h, h, True, pad=pad)
    k, v, kr = k[:9000], v[:9000], kr[:9000]
    cq, ck = cu_of(lq, dev), cu_of(lk, dev)
    md = mla.mla_get_metadata_prefill(cq, ck, 256, 9000, h, h)
    assert md[CUTS].item() > 0
    out, lse = unset(q)
    mla.mla_prefill(q, k, v, cq, ck, k_rope=kr, out=out, lse=lse, metadata=md)
    assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
    assert (out == 5).all() and (lse == 5).all()
    # the same partition in its own call, and the padded call with a partition of its own
    for x, mine in ((q[:256], md), (q, mla.mla_get_metadata_prefill(cq, ck, q.shape[0], 9000, h, h)), (q, None)):
        out, lse = unset(x)
        mla.mla_prefill(x, k, v, cq, ck, k_rope=kr, out=out, lse=lse, metadata=mine)
        check(out, lse, q, k, v, kr, lq, lk, True, heads=[0, 15])
        assert (out[256:] == 5).all() and (lse[256:] == 5).all()
    assert mla.mla_device_status() == 0


def test_cuts_that_a_call_of_fewer_keys_would_not_join(dev):
    """Made for a key tensor with a row behind the last sequence, used without that row, where so few keys are never cut."""
    lq, lk = [64], [1152]
    q, k, v, kr = make(dev, lq, lk, 2, 2, True)
    cq, ck = cu_of(lq, dev), cu_of(lk, dev)
    md = mla.mla_get_metadata_prefill(cq, ck, 64, 1153, 2, 2)
    assert md[CUTS].item() > 0
    out, lse = unset(q)
    mla.mla_prefill(q, k, v, cq, ck, k_rope=kr, out=out, lse=lse, metadata=md)
    assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
    assert (out == 5).all() and (lse == 5).all()
    mla.mla_prefill(q, k, v, cq, ck, k_rope=kr, out=out, lse=lse)
    check(out, lse, q, k, v, kr, lq, lk, True)


@pytest.mark.parametrize("lq,lk", [([70, 33], [70, 50]), ([64, 3], [9000, 40])])
def test_padded_rows_and_keys(dev, lq, lk):
    """Made for the rows alone, used with a few rows and keys behind them (and the other way round): the same outputs."""
    n, m, pad = sum(lq), sum(lk), 50
    q, k, v, kr = make(dev, lq, lk, 4, 2, True, pad=pad)
    cq, ck = cu_of(lq, dev), cu_of(lk, dev)
    want, want_lse = mla.mla_prefill(q[:n], k[:m], v[:m], cq, ck, k_rope=kr[:m])
    for made, used in ((0, pad), (pad, 0)):
        md = mla.mla_get_metadata_prefill(cq, ck, n + made, m + made, 4, 2)
        out, lse = unset(q[:n + used])
        mla.mla_prefill(q[:n + used], k[:m + used], v[:m + used], cq, ck, k_rope=kr[:m + used], out=out, lse=lse, metadata=md)
        assert torch.equal(out[:n], want) and torch.equal(lse[:n], want_lse)
        assert (out[n:] == 5).all() and (lse[n:] == 5).all()
    assert mla.mla_device_status() == 0
