"""Rows written into and read from the paged cache, and page keys, bit for bit against the definitions."""
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib
from tests import reference64 as R

pytestmark = pytest.mark.gpu
PAGE = 64
FORMATS = [("bf16", 576), ("bf16", 512), ("e4m3", 576)]


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_status_left():
    mla.mla_device_status()
    yield


def make(fmt, d, counts, starts, pad=0, seed=0, extra_pages=2):
    g = torch.Generator().manual_seed(seed)
    lens = [s + c for s, c in zip(starts, counts)]
    table, used = R.random_table(g, lens, nblk=sum((t + 63) // 64 for t in lens) + extra_pages)
    cu = torch.zeros((len(counts) + 1,), dtype=torch.int32)
    cu[1:] = torch.tensor(counts).cumsum(0)
    n = int(cu[-1]) + pad
    x = torch.randn((n, d), generator=g) * torch.exp(torch.randn((n, 1), generator=g))
    return R.random_cache(g, used, d, fmt == "e4m3"), table, cu, x.to(torch.bfloat16), lens


def written(cache, table, starts, counts, x, fmt):
    """The cache after the rows are written, by the definition."""
    want = cache.clone()
    r = 0
    d = x.shape[1]
    for b, c in enumerate(counts):
        for i in range(c):
            blk, off = R.place(table, b, starts[b] + i)
            if fmt == "bf16":
                want[blk, off, 0] = x[r]
            else:
                codes, s = R.quantised_row(x[r])
                want[blk, off * d:(off + 1) * d] = codes
                want[blk, PAGE * d + 4 * off:PAGE * d + 4 * off + 4] = s.reshape(1).view(torch.uint8)
            r += 1
    return want


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def write(fmt, latent, rope, cache, table, starts, cu=None):
    (mla.mla_cache_write_fp8 if fmt == "e4m3" else mla.mla_cache_write)(latent, rope, cache, table, starts, cu_rows=cu)


def read(fmt, *a, **k):
    return (mla.mla_cache_read_fp8 if fmt == "e4m3" else mla.mla_cache_read)(*a, **k)


def i32(v, dev):
    return torch.tensor(list(v), dtype=torch.int32, device=dev)


def parts(x, d):
    return x[:, :512], (x[:, 512:] if d > 512 else None)


@pytest.mark.parametrize("fmt,d", FORMATS)
@pytest.mark.parametrize("counts,starts,pad", [
    ([1], [0], 0), ([1, 1, 1], [63, 64, 0], 0), ([0, 1, 63, 64, 65], [5, 60, 1, 63, 0], 3),
    ([200, 0, 0, 7], [0, 9, 64, 130], 77), ([1] * 70, list(range(70)), 1), ([0, 0], [3, 4], 5)])
def test_write_and_read(dev, fmt, d, counts, starts, pad):
    cache, table, cu, x, _ = make(fmt, d, counts, starts, pad)
    want = written(cache, table, starts, counts, x, fmt)
    dc, dt, xd = cache.to(dev), table.to(dev), x.to(dev)
    lat, rope = parts(xd, d)
    write(fmt, lat, rope, dc, dt, i32(starts, dev), cu.to(dev))
    assert mla.mla_device_status() == 0
    assert torch.equal(bits(dc.cpu()), bits(want))
    # and back: every row of a sequence, nothing behind them
    out = torch.full((x.shape[0], d + 8), 7.0, dtype=torch.bfloat16, device=dev)
    lat, rope = out[:, :512], (out[:, 512:576] if d > 512 else None)
    read(fmt, dc, dt, i32(starts, dev), x.shape[0], cu_rows=cu.to(dev), latent=lat, k_rope=rope)
    assert mla.mla_device_status() == 0
    n = int(cu[-1])
    rows = R.cache_rows(want)
    got = out.cpu()
    assert bool((got[n:] == 7).all()) and bool((got[:, d:] == 7).all())
    r = 0
    for b, c in enumerate(counts):
        for i in range(c):
            blk, off = R.place(table, b, starts[b] + i)
            # scale * code has 28 bits: fp32 rounds it once, bf16 once more, as the definition does
            assert torch.equal(got[r, :d], R.f32(rows[blk, off]).to(torch.bfloat16)), (b, i)
            r += 1


@pytest.mark.parametrize("fmt,d", FORMATS)
def test_uniform_rows_without_offsets(dev, fmt, d):
    counts, starts = [3] * 5, [0, 62, 64, 100, 7]
    cache, table, cu, x, _ = make(fmt, d, counts, starts)
    want = written(cache, table, starts, counts, x, fmt)
    dc = cache.to(dev)
    xd = x.to(dev).contiguous()
    lat, rope = parts(xd, d)
    write(fmt, lat.contiguous(), None if rope is None else rope.contiguous(), dc, table.to(dev), i32(starts, dev))
    assert torch.equal(bits(dc.cpu()), bits(want))
    lat2, rope2 = read(fmt, dc, table.to(dev), i32(starts, dev), 15)
    lat3, rope3 = read(fmt, dc, table.to(dev), i32(starts, dev), 15, cu_rows=cu.to(dev))
    assert torch.equal(lat2, lat3) and (rope2 is None or torch.equal(rope2, rope3))
    assert (rope2 is None) == (d == 512)


def test_no_rows(dev):
    cache, table, cu, x, _ = make("bf16", 576, [0, 0], [3, 4])
    dc = cache.to(dev)
    lat, rope = parts(x.to(dev), 576)
    mla.mla_cache_write(lat, rope, dc, table.to(dev), i32([3, 4], dev), cu.to(dev))
    assert torch.equal(bits(dc.cpu()), bits(cache)) and mla.mla_device_status() == 0


def test_one_row_repeated(dev):
    """An expanded row (stride 0) is read for every position."""
    cache, table, cu, _, _ = make("bf16", 576, [70], [10])
    one = torch.randn((1, 576), dtype=torch.float32).to(torch.bfloat16)
    dc, x = cache.to(dev), one.to(dev).expand(70, 576)
    mla.mla_cache_write(x[:, :512], x[:, 512:], dc, table.to(dev), i32([10], dev), cu.to(dev))
    assert torch.equal(bits(dc.cpu()), bits(written(cache, table, [10], [70], one.expand(70, 576), "bf16")))


@pytest.mark.parametrize("fmt,d", [("bf16", 576), ("e4m3", 576)])
def test_many_sequences(dev, fmt, d):
    """More sequences than one level of the search covers, many of them without rows."""
    g = torch.Generator().manual_seed(4)
    counts = torch.randint(0, 3, (2500,), generator=g).tolist()
    counts[0] = counts[-1] = counts[1200] = 0
    starts = torch.randint(0, 40, (2500,), generator=g).tolist()
    cache, table, cu, x, _ = make(fmt, d, counts, starts, pad=11)
    dc = cache.to(dev)
    lat, rope = parts(x.to(dev), d)
    write(fmt, lat, rope, dc, table.to(dev), i32(starts, dev), cu.to(dev))
    assert mla.mla_device_status() == 0
    assert torch.equal(bits(dc.cpu()), bits(written(cache, table, starts, counts, x, fmt)))


def test_rows_that_do_not_fit_a_scale(dev):
    """Zeros, the smallest and largest values, NaN and infinities in the e4m3 cache."""
    x = torch.zeros((8, 576), dtype=torch.bfloat16)
    x[1] = torch.finfo(torch.bfloat16).tiny
    x[2, 5] = -3e-39                                  # below the normal range of bf16
    x[3] = torch.randn((576,)).to(torch.bfloat16)
    x[3, 7] = 114000.0                                # scale 254.46..
    x[4, 0] = 114240.0 * 2
    x[5, 575] = float("inf")
    x[6, 100] = float("nan")
    x[7] = torch.randn((576,)).to(torch.bfloat16)
    cache, table, cu, _, _ = make("e4m3", 576, [8], [60])
    want = written(cache, table, [60], [8], x, "e4m3")
    for rows, status in (([0, 1, 2, 3, 7], 0), ([4], _lib.MLA_DEVERR_SCALE), ([5], _lib.MLA_DEVERR_SCALE),
                         ([6], _lib.MLA_DEVERR_SCALE)):
        for r in rows:
            dc, xd = cache.to(dev), x[r:r + 1].to(dev)
            mla.mla_cache_write_fp8(xd[:, :512], xd[:, 512:], dc, table.to(dev), i32([60 + r], dev))
            assert mla.mla_device_status() == status, r
            blk, off = R.place(table, 0, 60 + r)
            got = dc.cpu()
            scale = got[blk, PAGE * 576 + 4 * off:PAGE * 576 + 4 * off + 4].clone().view(torch.float32)
            if r in (5, 6):
                assert torch.isnan(scale).all()
            else:
                assert torch.equal(got[blk, off * 576:(off + 1) * 576], want[blk, off * 576:(off + 1) * 576]), r
                assert torch.equal(scale, want[blk, PAGE * 576 + 4 * off:PAGE * 576 + 4 * off + 4].clone().view(torch.float32))


@pytest.mark.parametrize("fmt,d", FORMATS)
def test_places_that_do_not_exist(dev, fmt, d):
    """Positions outside the table and bad block ids are skipped and reported; the other rows are written."""
    counts, starts = [2, 2, 2], [0, 0, 0]
    cache, table, cu, x, _ = make(fmt, d, counts, starts)
    bad_table = table.clone()
    bad_table[1, 0] = cache.shape[0]
    lat, rope = parts(x.to(dev), d)
    width = table.shape[1] * 64
    for tb, st, status in ((table, [0, -1, 0], _lib.MLA_DEVERR_SEQLEN), (table, [0, width - 1, 0], _lib.MLA_DEVERR_SEQLEN),
                           (bad_table, [0, 0, 0], _lib.MLA_DEVERR_BLOCK_ID), (table, [0, 2 ** 31 - 1, 0], _lib.MLA_DEVERR_SEQLEN)):
        dc = cache.to(dev)
        write(fmt, lat, rope, dc, tb.to(dev), i32(st, dev), cu.to(dev))
        assert mla.mla_device_status() == status
        ok = [c if b != 1 else 0 for b, c in enumerate(counts)]
        skip = torch.cat([x[:2], x[4:]])
        want = written(cache, table, [0, 0, 0], ok, skip, fmt)
        if st[1] == -1:  # its second row is position 0
            blk, off = R.place(table, 1, 0)
            want = written(want, table[1:2], [0], [1], x[3:4], fmt)
        elif st[1] == width - 1:
            want = written(want, table[1:2], [width - 1], [1], x[2:3], fmt)
        assert torch.equal(bits(dc.cpu()), bits(want)), st
        out = torch.full((6, 576), 7.0, dtype=torch.bfloat16, device=dev)
        read(fmt, dc, tb.to(dev), i32(st, dev), 6, cu_rows=cu.to(dev), latent=out[:, :512],
             k_rope=out[:, 512:] if d > 512 else None)
        assert mla.mla_device_status() == status
        if st[1] not in (-1, width - 1):
            assert bool((out[2:4] == 7).all())


def test_offsets_past_32_bits(dev):
    """Pages whose byte and element offsets pass 2^32."""
    nblk = (2 ** 32) // (64 * 576) + 40          # 2^32 elements and a little: 8.6 GB
    cache = torch.empty((nblk, 64, 1, 576), dtype=torch.bfloat16, device=dev)
    cache[-2:] = 0
    cache[:2] = 0
    x = torch.randn((70, 576), device=dev).to(torch.bfloat16)
    table = torch.tensor([[nblk - 2, nblk - 1]], dtype=torch.int32, device=dev)
    mla.mla_cache_write(x[:, :512], x[:, 512:], cache, table, i32([0], dev))
    assert torch.equal(cache[-2:].view(128, 576)[:70], x) and not cache[:2].any() and not cache[-1, 6:].any()
    lat, rope = mla.mla_cache_read(cache, table, i32([0], dev), 70)
    assert torch.equal(torch.cat([lat, rope], 1), x)
    keys = torch.zeros((nblk, 576), dtype=torch.int8, device=dev)
    scales = torch.zeros((nblk,), device=dev)
    mla.mla_update_page_keys(cache, table, i32([70], dev), keys, scales)
    k, s = R.page_key(x[:64].cpu().double())
    assert torch.equal(keys[nblk - 2].cpu(), k) and float(scales[nblk - 2]) == s
    assert int((scales != 0).sum()) == 2 and mla.mla_device_status() == 0


def test_write_on_another_stream_and_in_a_graph(dev):
    counts, starts = [5, 0, 66], [61, 3, 0]
    cache, table, cu, x, _ = make("e4m3", 576, counts, starts)
    want = written(cache, table, starts, counts, x, "e4m3")
    dc, dt, cud, st = cache.to(dev), table.to(dev), cu.to(dev), i32(starts, dev)
    xd = torch.zeros_like(x, device=dev)
    s = torch.cuda.Stream(dev)
    with torch.cuda.stream(s):
        mla.mla_cache_write_fp8(xd[:, :512], xd[:, 512:], dc, dt, st, cud)
    s.synchronize()
    out = torch.zeros((x.shape[0], 576), dtype=torch.bfloat16, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_cache_write_fp8(xd[:, :512], xd[:, 512:], dc, dt, st, cud)
        mla.mla_cache_read_fp8(dc, dt, st, x.shape[0], cud, out[:, :512], out[:, 512:])
    xd.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dc.cpu(), want)
    rows = R.cache_rows(want)
    blk, off = R.place(table, 2, 65)
    assert torch.equal(out.cpu()[-1], R.f32(rows[blk, off]).to(torch.bfloat16))


# ---------------------------------------------------------------- page keys
def keys_of(cache, table, lens, starts, keys, scales):
    keys, scales = keys.clone(), scales.clone()
    rows = R.cache_rows(cache)
    for b, T in enumerate(lens):
        for pg in range((starts[b] if starts else 0) // 64, (T + 63) // 64):
            blk = int(table[b, pg])
            k, s = R.page_key(rows[blk, :min(64, T - 64 * pg)])
            keys[blk], scales[blk] = k, s
    return keys, scales


def update(fmt, *a, **k):
    (mla.mla_update_page_keys_fp8 if fmt == "e4m3" else mla.mla_update_page_keys)(*a, **k)


@pytest.mark.parametrize("fmt,d", FORMATS)
@pytest.mark.parametrize("lens,starts", [
    ([1], None), ([0, 1, 63, 64, 65, 130, 700], None), ([0, 1, 63, 64, 65, 130, 700], [0, 0, 62, 64, 63, 1, 699]),
    ([64 + i % 3 for i in range(600)], [64] * 600)])
def test_page_keys(dev, fmt, d, lens, starts):
    g = torch.Generator().manual_seed(9)
    table, used = R.random_table(g, lens, nblk=sum((t + 63) // 64 for t in lens) + 2, extra=3)
    cache = R.random_cache(g, used, d, fmt == "e4m3")
    keys = torch.full((used, d), 99, dtype=torch.int8)
    scales = torch.full((used,), -5.0)
    want = keys_of(cache, table, lens, starts, keys, scales)
    dk, ds = keys.to(dev), scales.to(dev)
    update(fmt, cache.to(dev), table.to(dev), i32(lens, dev), dk, ds, starts=None if starts is None else i32(starts, dev))
    assert mla.mla_device_status() == 0
    assert torch.equal(dk.cpu(), want[0]) and torch.equal(ds.cpu(), want[1])


@pytest.mark.parametrize("fmt,d", FORMATS)
def test_page_keys_of_unusual_rows(dev, fmt, d):
    """Zeros, NaN past the end (no part of the page), and NaN and infinities inside it."""
    g = torch.Generator().manual_seed(3)
    lens = [64, 30, 64, 64]
    table, used = R.random_table(g, lens)
    x = torch.randn((used, 64, d), generator=g)
    blk = [int(table[b, 0]) for b in range(4)]
    x[blk[0]] = 0
    from mla_decode_attention_latent_gb300 import workloads as W
    cache = W.pack_e4m3_pages(x) if fmt == "e4m3" else x[:, :, None].to(torch.bfloat16)

    def spoil(b, row, v):
        if fmt == "e4m3":
            cache[b, 64 * d + 4 * row:64 * d + 4 * row + 4] = torch.tensor([v]).view(torch.uint8)
        else:
            cache[b, row, 0, 3] = v
    spoil(blk[1], 30, float("nan"))
    spoil(blk[1], 63, float("inf"))
    spoil(blk[2], 0, float("nan"))
    spoil(blk[3], 63, float("inf"))
    want = keys_of(cache, table, lens, None, torch.zeros((used, d), dtype=torch.int8), torch.zeros((used,)))
    dk, ds = torch.full((used, d), 99, dtype=torch.int8, device=dev), torch.zeros((used,), device=dev)
    update(fmt, cache.to(dev), table.to(dev), i32(lens, dev), dk, ds)
    assert torch.equal(dk.cpu(), want[0])
    assert torch.equal(ds.cpu().nan_to_num(nan=-1), want[1].nan_to_num(nan=-1))
    assert float(ds[blk[0]]) == 1 and bool(torch.isnan(ds[[blk[2], blk[3]]]).all())


def test_page_keys_report_bad_lengths_and_blocks(dev):
    g = torch.Generator().manual_seed(3)
    table, used = R.random_table(g, [64, 64])
    cache = R.random_cache(g, used, 576, False).to(dev)
    for lens, tb, status in (([64, -1], table, _lib.MLA_DEVERR_SEQLEN), ([64, 65], table, _lib.MLA_DEVERR_SEQLEN),
                             ([64, 64], torch.tensor([[int(table[0, 0])], [-3]], dtype=torch.int32), _lib.MLA_DEVERR_BLOCK_ID)):
        keys, scales = torch.zeros((used, 576), dtype=torch.int8, device=dev), torch.zeros((used,), device=dev)
        mla.mla_update_page_keys(cache, tb.to(dev), i32(lens, dev), keys, scales)
        assert mla.mla_device_status() == status
        assert float(scales[int(table[0, 0])]) > 0


@pytest.mark.parametrize("exponent", [40, 120, 127, 134, 140])
def test_codes_of_every_value(dev, exponent):
    """Every significand of the row's largest value with every bf16 value of the 12 octaves below it, among them all
    quotients that lie on or next to a rounding border: the codes are those of the division."""
    amax = torch.tensor([(exponent << 7) | m for m in range(128)], dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    values = torch.arange((exponent - 12) << 7, (exponent + 1) << 7, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    rows = []
    for m in range(128):
        v = values[values.float() <= amax[m].float()]
        v = torch.cat([v, -v])
        v = torch.cat([v, v[:(-v.numel()) % 575]]).view(-1, 575)
        rows.append(torch.cat([amax[m].expand(v.shape[0], 1), v], 1))
    x = torch.cat(rows)
    blocks = (x.shape[0] + 63) // 64
    cache = torch.zeros((blocks, _lib.MLA_FP8_PAGE_BYTES(576)), dtype=torch.uint8, device=dev)
    xd = x.to(dev)
    mla.mla_cache_write_fp8(xd[:, :512], xd[:, 512:], cache, torch.arange(blocks, dtype=torch.int32, device=dev)[None],
                            i32([0], dev))
    scale = x[:, 0].float() / torch.tensor(448.0)
    want = (x.float() / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    got = cache.cpu()
    assert torch.equal(got[:, 64 * 576:].contiguous().view(torch.float32).view(-1)[:x.shape[0]], scale)
    assert torch.equal(got[:, :64 * 576].reshape(-1, 576)[:x.shape[0]], want)
    assert mla.mla_device_status() in (0, _lib.MLA_DEVERR_SCALE)
