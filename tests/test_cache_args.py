"""The cache, page-selection and draft-tree calls refuse bad arguments on the host, before anything is launched."""
import numpy as np
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib
from mla_decode_attention_latent_gb300 import build as cuda_build
from tests import reference64 as R

BAD, UNSUP, WS = _lib.MLA_ERR_INVALID_ARG, _lib.MLA_ERR_UNSUPPORTED, _lib.MLA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return _lib.load()


def rows(lib, fp8=False, read=False, **over):
    a = dict(latent=256, ls=576, rope=256, rs=576, n=8, cu=256, starts=256, b=4, cache=256, nblk=4, bt=256, mb=2, d=576)
    a.update(over)
    if read:
        call = lib.mla_cache_read_fp8 if fp8 else lib.mla_cache_read
        return call(a["cache"], a["nblk"], a["bt"], a["mb"], a["starts"], a["cu"], a["b"], a["n"], a["latent"], a["ls"],
                    a["rope"], a["rs"], a["d"], None)
    call = lib.mla_cache_write_fp8 if fp8 else lib.mla_cache_write
    return call(a["latent"], a["ls"], a["rope"], a["rs"], a["n"], a["cu"], a["starts"], a["b"], a["cache"], a["nblk"],
                a["bt"], a["mb"], a["d"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(latent=None), BAD), (dict(rope=None), BAD), (dict(starts=None), BAD), (dict(cache=None), BAD), (dict(bt=None), BAD),
    (dict(b=0), BAD), (dict(n=-1), BAD), (dict(nblk=0), BAD), (dict(mb=0), BAD), (dict(d=0), BAD),
    (dict(latent=264), BAD), (dict(rope=264), BAD), (dict(cache=264), BAD),       # not 16-byte aligned
    (dict(ls=580), BAD), (dict(rs=68), BAD), (dict(ls=-8), BAD),
    (dict(cu=None, n=9), BAD),                                                    # 4 sequences, 9 rows
    (dict(mb=1 << 25), BAD), (dict(n=1 << 31), UNSUP), (dict(d=448), UNSUP)])
def test_rows(lib, fp8, read, over, code):
    assert rows(lib, fp8, read, **over) == code


def test_rows_of_one_format_only(lib):
    assert rows(lib, True, d=512) == UNSUP and rows(lib, True, True, d=512) == UNSUP
    # overlapping rows may be read by a write, never written by a read
    assert rows(lib, read=True, ls=504) == BAD and rows(lib, read=True, rs=56) == BAD
    # nothing to do: no launch, so no device is needed
    for fp8 in (False, True):
        for read in (False, True):
            assert rows(lib, fp8, read, n=0) == _lib.MLA_OK
            assert rows(lib, fp8, read, n=0, latent=None, rope=None) == _lib.MLA_OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(cache=None), BAD), (dict(bt=None), BAD), (dict(sl=None), BAD), (dict(keys=None), BAD), (dict(scales=None), BAD),
    (dict(b=0), BAD), (dict(nblk=0), BAD), (dict(mb=0), BAD), (dict(keys=264), BAD), (dict(cache=264), BAD), (dict(d=448), UNSUP)])
def test_page_keys(lib, fp8, over, code):
    a = dict(cache=256, nblk=4, bt=256, mb=2, sl=256, starts=None, b=2, d=576, keys=256, scales=256)
    a.update(over)
    call = lib.mla_update_page_keys_fp8 if fp8 else lib.mla_update_page_keys
    assert call(a["cache"], a["nblk"], a["bt"], a["mb"], a["sl"], a["starts"], a["b"], a["d"], a["keys"], a["scales"], None) == code


def blocks(lib, fp8=False, **over):
    a = dict(q=256, cache=256, nblk=4, bt=256, mb=9, sl=256, keys=256, scales=256, topk=4, sink=1, local=1, b=2, s=1, h=16,
             hkv=1, d=576, dv=512, parts=3, scale=1 / 24, causal=0, o=256, lse=256, pages=256, ws=256, bytes=1 << 30)
    a.update(over)
    call = lib.mla_decode_kvcache_blocks_fp8 if fp8 else lib.mla_decode_kvcache_blocks
    return call(*[a[k] for k in ("q", "cache", "nblk", "bt", "mb", "sl", "keys", "scales", "topk", "sink", "local", "b", "s",
                                 "h", "hkv", "d", "dv", "parts", "scale", "causal", "o", "lse", "pages", "ws", "bytes")], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over,code", [
    *[({k: None}, BAD) for k in ("q", "cache", "bt", "sl", "keys", "scales", "o", "lse", "pages", "ws")],
    *[({k: 0}, BAD) for k in ("nblk", "mb", "topk", "local", "b", "s", "h", "hkv", "d", "dv", "parts")],
    (dict(sink=-1), BAD), (dict(sink=4, local=1), BAD), (dict(sink=1, local=4), BAD), (dict(sink=2 ** 31 - 1, local=2 ** 31 - 1), BAD),
    (dict(scale=0.0), BAD), (dict(scale=-0.1), BAD), (dict(scale=float("nan")), BAD),
    (dict(q=264), BAD), (dict(keys=264), BAD), (dict(o=264), BAD), (dict(ws=272), BAD), (dict(mb=1 << 25), BAD),
    (dict(dv=256), UNSUP), (dict(hkv=2), UNSUP), (dict(d=448), UNSUP), (dict(b=65536), UNSUP), (dict(b=8192, s=8), UNSUP),
    (dict(h=16385), UNSUP), (dict(topk=1 << 25), UNSUP), (dict(bytes=4096), WS)])
def test_blocks(lib, fp8, over, code):
    assert blocks(lib, fp8, **over) == code


def test_blocks_workspace(lib):
    n = lib.mla_blocks_workspace_bytes(4, 2, 128, 1, 512, 100, 16, 76)
    decode = (8 + 76) * 128 * 513 * 4
    assert n % 256 == 0 and n >= decode + 4 * 8 * 100 + 4 * 8 * 16 + 4 * 8 + 32 * 76 + 4 * 9
    for bad in ((0, 2, 128, 1, 512, 100, 16, 76), (4, 0, 128, 1, 512, 100, 16, 76), (4, 2, 0, 1, 512, 100, 16, 76),
                (4, 2, 128, 2, 512, 100, 16, 76), (4, 2, 128, 1, 576, 100, 16, 76), (4, 2, 128, 1, 512, 0, 16, 76),
                (4, 2, 128, 1, 512, 100, 0, 76), (4, 2, 128, 1, 512, 100, 16, 0), (65535, 2, 128, 1, 512, 100, 16, 76)):
        assert lib.mla_blocks_workspace_bytes(*bad) == 0
    # one byte short is refused
    assert blocks(lib, b=4, s=2, h=128, mb=100, topk=16, parts=76, bytes=n - 1) == WS


def tree(lib, fp8=False, **over):
    a = dict(q=256, cache=256, nblk=4, bt=256, mb=9, sl=256, mask=256, lens=None, b=2, s=4, h=16, hkv=1, d=576, dv=512, md=256,
             ns=256, parts=3, scale=1 / 24, o=256, lse=256, ws=256, bytes=1 << 30)
    a.update(over)
    call = lib.mla_decode_kvcache_tree_fp8 if fp8 else lib.mla_decode_kvcache_tree
    return call(*[a[k] for k in ("q", "cache", "nblk", "bt", "mb", "sl", "mask", "lens", "b", "s", "h", "hkv", "d", "dv", "md",
                                 "ns", "parts", "scale", "o", "lse", "ws", "bytes")], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over,code", [
    *[({k: None}, BAD) for k in ("q", "cache", "bt", "sl", "mask", "md", "ns", "o", "lse", "ws")],
    # without a partition (the call makes its own) the same are refused, before it is launched
    *[({k: None, "md": None, "ns": None}, BAD) for k in ("q", "cache", "bt", "sl", "mask", "o", "lse", "ws")],
    *[({k: 0, "md": None, "ns": None}, BAD) for k in ("nblk", "mb", "b", "s", "h", "hkv", "d", "dv", "parts")],
    *[({**v, "md": None, "ns": None}, c) for v, c in ((dict(scale=float("nan")), BAD), (dict(q=264), BAD), (dict(dv=256), UNSUP),
                                                       (dict(hkv=2), UNSUP), (dict(d=448), UNSUP), (dict(s=8192, h=16), UNSUP),
                                                       (dict(mb=1 << 25), BAD), (dict(b=65536), BAD), (dict(bytes=4096), WS))],
    *[({k: 0}, BAD) for k in ("nblk", "mb", "b", "s", "h", "hkv", "d", "dv", "parts")],
    (dict(scale=float("nan")), BAD), (dict(q=264), BAD), (dict(dv=256), UNSUP), (dict(hkv=2), UNSUP), (dict(d=448), UNSUP),
    (dict(s=8192, h=16), UNSUP), (dict(bytes=4096), WS)])
def test_tree(lib, fp8, over, code):
    assert tree(lib, fp8, **over) == code


def test_e4m3_calls_take_576_wide_rows_only(lib):
    assert tree(lib, True, d=512) == UNSUP and blocks(lib, True, d=512) == UNSUP


@pytest.mark.parametrize("args,code", [((None, 2, 4, 256), BAD), ((256, 0, 4, 256), BAD), ((256, 2, 0, 256), BAD),
                                       ((256, 2, 4, None), BAD), ((256, 1, 65537, 256), UNSUP), ((256, 1 << 20, 4096, 256), UNSUP)])
def test_tree_mask(lib, args, code):
    assert lib.mla_tree_mask(*args, None) == code


def test_tensors_of_the_host_are_refused():
    x, cache = torch.zeros((4, 576), dtype=torch.bfloat16), torch.zeros((2, 64, 1, 576), dtype=torch.bfloat16)
    table, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1,), dtype=torch.int32)
    keys, scales = torch.zeros((2, 576), dtype=torch.int8), torch.zeros((2,))
    q = torch.zeros((1, 1, 16, 576), dtype=torch.bfloat16)
    for call in (lambda: mla.mla_cache_write(x[:, :512], x[:, 512:], cache, table, n),
                 lambda: mla.mla_cache_read(cache, table, n, 4),
                 lambda: mla.mla_update_page_keys(cache, table, n, keys, scales),
                 lambda: mla.mla_decode_kvcache_blocks(q, cache, table, n, keys, scales, 2, 512),
                 lambda: mla.mla_decode_kvcache_tree(q, cache, table, n, n.view(1, 1, 1), 512),
                 lambda: mla.mla_tree_mask(table)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_rows_that_are_not_a_matrix_are_refused():
    cache, table = torch.zeros((2, 64, 1, 576), dtype=torch.bfloat16), torch.zeros((1, 2), dtype=torch.int32)
    for call in (mla.mla_cache_write, mla.mla_cache_write_fp8):
        with pytest.raises(TypeError, match="torch.Tensor"):
            call([[0.0] * 512], None, cache, table, table[:, 0])
        for shape in ((), (512,), (1, 1, 512)):
            with pytest.raises(ValueError, match="latent must be"):
                call(torch.zeros(shape, dtype=torch.bfloat16), None, cache, table, table[:, 0])


# ---------------------------------------------------------------- the tests' own restatements
def test_page_key_of_known_pages():
    rows = torch.zeros((2, 4), dtype=torch.float64)
    rows[0] = torch.tensor([1.0, -2.0, 0.5, 0.0])
    rows[1] = torch.tensor([3.0, -2.0, 0.25, 0.0])
    key, scale = R.page_key(rows)
    assert scale == float(np.float32(2) / np.float32(127)) and key.tolist() == [127, -127, 24, 0]
    key, scale = R.page_key(torch.zeros((64, 4), dtype=torch.float64))
    assert scale == 1.0 and not key.any()


def test_selection_of_known_scores():
    score = torch.tensor([9.0, 1.0, 5.0, 5.0, float("nan"), 5.0, -1.0, 0.0])
    assert R.select(score, 8, 8, 1, 1) == list(range(8))
    assert R.select(score, 8, 5, 1, 1) == [0, 2, 3, 4, 7]
    assert R.select(score, 8, 2, 1, 1) == [0, 7]
    assert R.select(score, 8, 4, 0, 2) == [0, 4, 6, 7]


def test_mask_words_of_a_known_tree():
    assert R.mask_words(R.ancestors([-1, 0, 0, 2])).tolist() == [[1], [3], [5], [13]]
    assert R.mask_words(R.ancestors(list(range(-1, 31)) + [31]))[32].tolist() == [-1, 1]


def test_tree_partition(lib):
    for args, code in (((None, None, 2, 4, 16, 1, 3, 256, 256), BAD), ((256, None, 2, 4, 16, 1, 3, None, 256), BAD),
                       ((256, None, 2, 4, 16, 1, 3, 256, None), BAD), ((256, None, 0, 4, 16, 1, 3, 256, 256), BAD),
                       ((256, None, 2, 0, 16, 1, 3, 256, 256), BAD), ((256, None, 2, 4, 0, 1, 3, 256, 256), BAD),
                       ((256, None, 2, 4, 16, 1, 0, 256, 256), BAD), ((256, None, 2, 4, 16, 2, 3, 256, 256), UNSUP),
                       ((256, None, 2, 8192, 16, 1, 3, 256, 256), UNSUP), ((256, None, 65535, 512, 128, 1, 3, 256, 256), UNSUP)):
        assert lib.mla_get_metadata_tree(*args, None) == code
    # a slot holds one 128-row tile: 3 tiles of 2 sequences, 5 parts
    n = lib.mla_tree_workspace_bytes(2, 3, 100, 1, 512, 5)
    assert n % 256 == 0 and n >= (2 * 3 + 5) * 128 * 513 * 4 + 5 * 32 + 7 * 4 > n - 1024
    for bad in ((0, 3, 100, 1, 512, 5), (2, 0, 100, 1, 512, 5), (2, 3, 0, 1, 512, 5), (2, 3, 100, 2, 512, 5),
                (2, 3, 100, 1, 576, 5), (2, 3, 100, 1, 512, 0), (2, 8192, 16, 1, 512, 5), (65535, 512, 128, 1, 512, 5)):
        assert lib.mla_tree_workspace_bytes(*bad) == 0
    assert tree(lib, b=2, s=3, h=100, parts=5, md=None, ns=None, bytes=n - 1) == WS
    assert tree(lib, b=65535, s=512, h=128) == UNSUP
