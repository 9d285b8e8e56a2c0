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
