"""The arithmetic behind the e4m3 decodes' bound: what two 8-bit parts hold of a weight."""
import torch


def test_two_parts_hold_every_weight():
    """For every f16 value w up to 448: h = e4m3(w), l = e5m2(w - h); w - h is an f16, and h + l is off by at most
    2^-8 of w, or 2^-14 where that is more."""
    w = torch.arange(0, 0x7c00, dtype=torch.int32).to(torch.int16).view(torch.float16)
    w = w[w <= 448]
    h = w.to(torch.float8_e4m3fn).float()
    rest = w.float() - h
    assert torch.equal(rest.to(torch.float16).float(), rest)
    error = (rest - rest.to(torch.float8_e5m2).float()).abs()
    assert bool((error <= torch.clamp(w.float() * 2.0 ** -8, min=2.0 ** -14)).all())
