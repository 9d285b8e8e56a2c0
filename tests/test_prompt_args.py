"""The prompt path's calls refuse bad arguments on the host, before anything is launched."""
import ctypes

import pytest

from mla_decode_attention_latent_gb300 import _lib
from mla_decode_attention_latent_gb300 import build as cuda_build

BAD, UNSUP, WS, OK = _lib.MLA_ERR_INVALID_ARG, _lib.MLA_ERR_UNSUPPORTED, _lib.MLA_ERR_WORKSPACE, _lib.MLA_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return _lib.load()


def call(fn, defaults, over):
    a = dict(defaults)
    a.update(over)
    return fn(*a.values(), None)


ASSIGN = dict(sl=256, cu=256, b=4, n=8, bt=256, mb=2, free=256, cap=9, left=256, left_out=256, new=256, pos=256, slots=256)


@pytest.mark.parametrize("over,code", [
    *[({k: None}, BAD) for k in ("sl", "cu", "bt", "free", "left", "left_out", "new")],
    *[({k: 0}, BAD) for k in ("b", "mb", "cap")], (dict(n=-1), BAD), (dict(mb=1 << 25), BAD), (dict(n=1 << 31), UNSUP), (dict(cap=1 << 31), UNSUP)])
def test_assign(lib, over, code):
    assert call(lib.mla_assign_pages, ASSIGN, over) == code


@pytest.mark.parametrize("over,code", [
    *[({k: None}, BAD) for k in ("sl", "done", "bt", "free", "left")], *[({k: 0}, BAD) for k in ("b", "mb", "nblk", "cap")], (dict(mb=1 << 25), BAD),
    (dict(cap=1 << 31), UNSUP)])
def test_release(lib, over, code):
    assert call(lib.mla_release_pages, dict(sl=256, done=256, b=4, bt=256, mb=2, nblk=9, free=256, cap=9, left=256), over) == code


@pytest.mark.parametrize("over,code", [
    ({}, OK), (dict(dims=0), BAD), (dict(dims=63), BAD), (dict(dims=-2), BAD), (dict(base=1.0), BAD), (dict(base=NAN), BAD), (dict(base=INF), BAD),
    (dict(factor=0.5), BAD), (dict(factor=NAN), BAD), (dict(factor=INF), BAD), (dict(original=-1), BAD), (dict(original=4096, fast=0.5), BAD),
    (dict(original=4096, slow=0.0), BAD), (dict(original=4096, fast=INF), BAD), (dict(original=4096, fast=NAN), BAD), (dict(original=4096), OK)])
def test_turns(lib, over, code):
    a = dict(dims=64, base=10000.0, factor=4.0, original=0, fast=32.0, slow=1.0)
    a.update(over)
    assert lib.mla_rope_turns(*a.values(), (ctypes.c_int64 * 64)()) == code
    assert lib.mla_rope_turns(64, 1e4, 1.0, 0, 32.0, 1.0, None) == BAD


HEADS = dict(x=256, xt=192 * 16, xh=192, n=7, h=16, d=192, w=256, eps=1e-6, pos=256, turns=256, dims=64, il=0, scale=1.0, out=512, ot=192 * 16, oh=192)


@pytest.mark.parametrize("over,code", [
    *[({k: None}, BAD) for k in ("x", "out", "pos", "turns")], (dict(n=-1), BAD), (dict(h=0), BAD), (dict(d=0), BAD), (dict(dims=-16), BAD),
    (dict(d=188), UNSUP), (dict(d=584), UNSUP), (dict(dims=24), UNSUP), (dict(dims=208), UNSUP), (dict(d=576, dims=272), UNSUP),
    (dict(n=1 << 31), UNSUP), (dict(n=(1 << 31) - 1, h=1 << 10), UNSUP),
    (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
    (dict(x=264), BAD), (dict(out=264), BAD), (dict(w=264), BAD), (dict(xt=190), BAD), (dict(xh=190), BAD), (dict(ot=190), BAD), (dict(oh=190), BAD),
    (dict(xh=-8), BAD), (dict(oh=184), BAD), (dict(ot=192 * 15), BAD), (dict(ot=0), BAD), (dict(oh=0), BAD),  # written heads would overlap
    (dict(out=256, oh=200, ot=200 * 16), BAD),  # in place with other strides
    (dict(n=0), OK), (dict(n=0, x=None, out=None, pos=None, turns=None), OK), (dict(out=256, w=None, dims=0, pos=None, turns=None), OK)])
def test_heads(lib, over, code):
    assert call(lib.mla_norm_rope, HEADS, over) == code


ROWS = dict(latent=256, ls=576, rope=256, rs=576, n=8, w=256, eps=1e-6, pos=256, turns=256, il=0, scale=1.0, slots=256, cache=256, nblk=4, d=576, lo=None,
            los=0, ro=None, ros=0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over,code", [
    *[({k: None}, BAD) for k in ("latent", "rope", "pos", "turns", "slots", "cache")], (dict(n=-1), BAD), (dict(nblk=0), BAD), (dict(d=0), BAD),
    (dict(d=448), UNSUP), (dict(n=1 << 31), UNSUP), (dict(nblk=1 << 31), UNSUP), (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(scale=INF), BAD),
    (dict(latent=264), BAD), (dict(rope=264), BAD), (dict(cache=264), BAD), (dict(w=264), BAD), (dict(ls=580), BAD), (dict(rs=68), BAD), (dict(ls=-8), BAD),
    (dict(lo=264, los=512), BAD), (dict(lo=256, los=504), BAD), (dict(ro=256, ros=56), BAD), (dict(ro=264, ros=64), BAD),
    (dict(n=0), OK), (dict(n=0, latent=None, rope=None, pos=None, turns=None, slots=None), OK)])
def test_rows(lib, fp8, over, code):
    assert call(lib.mla_norm_rope_cache_write_fp8 if fp8 else lib.mla_norm_rope_cache_write, ROWS, over) == code


def test_rows_of_one_format_only(lib):
    assert call(lib.mla_norm_rope_cache_write_fp8, ROWS, dict(d=512)) == UNSUP
    assert call(lib.mla_norm_rope_cache_write, ROWS, dict(d=512, ro=256, ros=64)) == BAD  # no RoPE part to write
    assert call(lib.mla_norm_rope_cache_write, ROWS, dict(d=512, n=0)) == OK


PREFILL = dict(q=256, qt=16 * 192, qh=192, k=256, kt=4 * 256, kh=256, v=512, vt=4 * 256, vh=256, kr=256, krt=64, cq=256, ck=256, b=2, nq=9, nk=11, hq=16, hkv=4, dqk=192,
               dv=128, scale=0.07, causal=1, md=256, out=512, lse=256, ws=256, bytes=1 << 40)


@pytest.mark.parametrize("over,code", [
    *[({k: None}, BAD) for k in ("q", "k", "v", "kr", "cq", "ck", "out", "lse", "ws")],
    *[({k: 0}, BAD) for k in ("b", "hq", "hkv", "dqk", "dv")], (dict(nq=-1), BAD), (dict(nk=-1), BAD), (dict(hq=18), BAD),
    (dict(hq=129 * 4), UNSUP), (dict(hq=4096 * 8, hkv=4096), UNSUP), (dict(nq=1 << 30), UNSUP), (dict(nk=1 << 30), UNSUP),
    (dict(dqk=160), UNSUP), (dict(dqk=576), UNSUP), (dict(dv=64), UNSUP), (dict(dqk=128), BAD),  # a RoPE key with heads that have no room for it
    (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD), (dict(scale=3.4e38), BAD),
    (dict(q=264), BAD), (dict(k=264), BAD), (dict(v=264), BAD), (dict(kr=264), BAD), (dict(out=528), BAD), (dict(ws=384), BAD),
    (dict(qt=3076), BAD), (dict(qh=190), BAD), (dict(kt=8), BAD), (dict(kh=120), BAD), (dict(vh=0), BAD), (dict(krt=56), BAD), (dict(krt=68), BAD),
    (dict(kt=1 << 40), BAD), (dict(nq=0), OK), (dict(nq=0, q=None, out=None, lse=None, ws=None), OK)])
def test_prefill(lib, over, code):
    assert call(lib.mla_prefill, PREFILL, over) == code


@pytest.mark.parametrize("over,code", [
    *[({k: None}, BAD) for k in ("cq", "ck", "md")], *[({k: 0}, BAD) for k in ("b", "hq", "hkv")], (dict(nq=-1), BAD), (dict(nk=-1), BAD), (dict(hq=18), BAD),
    (dict(hq=129 * 4), UNSUP), (dict(nq=1 << 30), UNSUP), (dict(nk=1 << 30), UNSUP)])
def test_prefill_partition(lib, over, code):
    assert call(lib.mla_get_metadata_prefill, dict(cq=256, ck=256, b=2, nq=9, nk=11, hq=16, hkv=4, causal=1, md=256), over) == code


def test_prefill_sizes_of_impossible_shapes(lib):
    for shape in ((0, 9, 16, 4), (2, -1, 16, 4), (2, 9, 18, 4), (2, 9, 0, 4), (2, 9, 516, 4), (2, 1 << 30, 16, 4)):
        assert lib.mla_prefill_metadata_ints(*shape) == 0 and lib.mla_prefill_workspace_bytes(*shape) == 0


def test_the_binding_refuses_host_tensors_and_wrong_kinds():
    import torch

    import mla_decode_attention_latent_gb300 as mla
    i, f, h, l = (torch.zeros((4,), dtype=t) for t in (torch.int32, torch.float32, torch.bfloat16, torch.int64))
    heads = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.mla_norm_rope(heads, None, None, weight=h)
    with pytest.raises(TypeError):
        mla.mla_norm_rope(heads.float(), None, None)
    with pytest.raises(TypeError):
        mla.mla_norm_rope([1], None, None)
    with pytest.raises(ValueError):
        mla.mla_assign_pages(i, i, torch.zeros((3, 2), dtype=torch.int32), i, i[:1], 4)
    with pytest.raises(ValueError):
        mla.mla_release_pages(i, i, torch.zeros((4, 2), dtype=torch.int32), 9, i, i[:1])
    with pytest.raises(ValueError):
        mla.mla_norm_rope_cache_write(torch.zeros((4, 512), dtype=torch.bfloat16), torch.zeros((4, 64), dtype=torch.bfloat16), i, l, l,
                                      torch.zeros((2, 64, 1, 576), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mla.mla_prefill(heads, heads, heads, i, i)
    with pytest.raises(ValueError):
        mla.mla_get_metadata_prefill(i, i, 4, 4, 2, 2)
    for dims in (0, -2, 7):
        with pytest.raises((ValueError, RuntimeError)):
            mla.mla_rope_turns(dims, device="cpu")
    with pytest.raises(RuntimeError):
        mla.mla_rope_turns(64, base=0.5, device="cpu")
    assert f.dtype == torch.float32
