"""The decode over selected pages: the selection page for page, the attention against 64 bits."""
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib
from tests import reference64 as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_status_left():
    mla.mla_device_status()
    yield


def make(lens, s_q, h, d=576, fp8=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    table, used = R.random_table(g, lens, extra=1)
    cache = R.random_cache(g, used, d, fp8)
    q = torch.randn((len(lens), s_q, h, d), generator=g).to(torch.bfloat16)
    keys = torch.randint(-127, 128, (used, d), generator=g).to(torch.int8)
    scales = torch.rand((used,), generator=g) + 0.5
    return q, cache, table, keys, scales


def reference(q, cache, table, lens, keys, scales, topk, sink, local, causal, scale):
    b, s_q, h, d = q.shape
    rows = R.cache_rows(cache)
    o = torch.zeros((b, s_q, h, 512), dtype=torch.float64)
    a, lse = o.clone(), torch.zeros((b, s_q, h), dtype=torch.float64)
    pages = torch.full((b, s_q, topk), -1, dtype=torch.int32)
    for i in range(b):
        for j in range(s_q):
            L = R.token_len(lens[i], s_q, j, causal)
            n = (L + 63) // 64
            blk = table[i, :n].long()
            pick = R.select(R.page_scores(q[i, j], keys[blk], scales[blk]) if n else torch.zeros(0), n, topk, sink, local)
            pages[i, j, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
            k = [rows[int(table[i, p])][:min(64, L - 64 * p)] for p in pick]
            k = torch.cat(k) if k else torch.zeros((0, d), dtype=torch.float64)
            o[i, j], lse[i, j], a[i, j] = R.attend(q[i, j], k, scale, cache.dtype != torch.bfloat16)
    return o, lse, a, pages


def decode(dev, q, cache, table, lens, keys, scales, topk, **k):
    call = mla.mla_decode_kvcache_blocks if cache.dtype == torch.bfloat16 else mla.mla_decode_kvcache_blocks_fp8
    return call(q.to(dev), cache.to(dev), table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), keys.to(dev),
                scales.to(dev), topk, 512, **k)


def check(dev, q, cache, table, lens, keys, scales, topk, sink=1, local=1, causal=False, status=0):
    scale = q.shape[3] ** -0.5
    ref = reference(q, cache, table, lens, keys, scales, topk, sink, local, causal, scale)
    o, lse, pages = decode(dev, q, cache, table, lens, keys, scales, topk, sink_pages=sink, local_pages=local, causal=causal)
    assert mla.mla_device_status() == status
    assert torch.equal(pages.cpu(), ref[3])
    R.assert_attention(o, lse, ref[0], ref[1], ref[2], cache.dtype != torch.bfloat16)
    return o, lse, pages


@pytest.mark.parametrize("d,fp8", [(576, False), (512, False), (576, True)])
@pytest.mark.parametrize("h", [1, 16, 100, 128, 160])
def test_heads(dev, d, fp8, h):
    lens = [1000, 0, 1, 64, 65, 700]
    check(dev, *make(lens, 1, h, d, fp8)[:3], lens, *make(lens, 1, h, d, fp8)[3:], topk=5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("s_q,lens", [(3, [400, 2, 66, 130, 0, 321]), (8, [515, 5, 900])])
def test_tokens(dev, fp8, causal, s_q, lens):
    q, cache, table, keys, scales = make(lens, s_q, 32, 576, fp8)
    check(dev, q, cache, table, lens, keys, scales, 4, causal=causal)


@pytest.mark.parametrize("topk,sink,local", [(1, 0, 1), (2, 1, 1), (2, 0, 1), (6, 3, 3), (7, 2, 4), (40, 1, 1), (33, 0, 2), (200, 1, 1)])
def test_forced_pages(dev, topk, sink, local):
    lens = [64 * 40, 64 * 33 + 1, 63]
    q, cache, table, keys, scales = make(lens, 1, 16)
    check(dev, q, cache, table, lens, keys, scales, topk, sink, local)


def test_long_sequences_with_many_ties(dev):
    """More pages than one round of the selection holds; a third of them share one key."""
    lens = [64 * 700 + 3, 64 * 300, 64 * 257]
    q, cache, table, keys, scales = make(lens, 1, 4)
    shared = torch.arange(keys.shape[0]) % 3 == 0
    keys[shared], scales[shared] = keys[0].clone(), 1.0
    check(dev, q, cache, table, lens, keys, scales, 190)
    check(dev, q, cache, table, lens, keys, scales, 300)


def test_largest_products_are_exact(dev):
    """Codes and queries at +-127 in every place: sums of 576 * 127^2 and their neighbours, one step apart."""
    lens = [64 * 130]
    q, cache, table, keys, scales = make(lens, 1, 16)
    keys[:] = 127
    for p in range(130):  # page p is p % 7 steps below the top
        keys[table[0, p].long(), :p % 7] = 126
    scales[:] = 1.0
    q[:] = 1.0
    check(dev, q, cache, table, lens, keys, scales, 60)
    q[:] = -1.0           # every score negative: the least negative first
    check(dev, q, cache, table, lens, keys, scales, 60)
    keys[:] = -keys
    check(dev, q, cache, table, lens, keys, scales, 60)


def test_zero_query_and_zero_keys(dev):
    lens = [64 * 20]
    q, cache, table, keys, scales = make(lens, 1, 16)
    q[:, :, :8] = 0
    check(dev, q, cache, table, lens, keys, scales, 6)
    q[:] = 0              # every page ties: the first ones
    _, _, pages = check(dev, q, cache, table, lens, keys, scales, 6)
    assert pages[0, 0].tolist() == [0, 1, 2, 3, 4, 19]


def test_scores_that_are_not_finite(dev):
    """A page without a finite mean is selected first; a query that is not finite ties every page."""
    lens = [64 * 20]
    q, cache, table, keys, scales = make(lens, 1, 16)
    for p in (7, 12):
        keys[table[0, p].long()], scales[table[0, p].long()] = 0, float("nan")
    _, _, pages = check(dev, q, cache, table, lens, keys, scales, 4)
    assert pages[0, 0].tolist() == [0, 7, 12, 19]
    for bad in (float("nan"), float("inf")):
        z = q.clone()
        z[0, 0, 3, 9] = bad
        _, _, pages = decode(dev, z, cache, table, lens, keys, scales, 4)
        assert pages[0, 0].tolist() == [0, 1, 2, 19]


def test_keys_that_the_library_keeps(dev):
    """write -> page keys -> selection -> decode, and the whole set of pages equals the dense decode."""
    lens = [64 * 9 + 5, 64 * 12, 40]
    g = torch.Generator().manual_seed(5)
    table, used = R.random_table(g, lens)
    q = torch.randn((3, 1, 128, 576), generator=g).to(torch.bfloat16).to(dev)
    x = torch.randn((sum(lens), 576), generator=g).to(torch.bfloat16)
    cu = torch.tensor([0, lens[0], lens[0] + lens[1], sum(lens)], dtype=torch.int32, device=dev)
    zero, sl, tb, xd = torch.zeros((3,), dtype=torch.int32, device=dev), torch.tensor(lens, dtype=torch.int32, device=dev), table.to(dev), x.to(dev)
    for fp8 in (False, True):
        cache = torch.zeros((used, _lib.MLA_FP8_PAGE_BYTES(576)), dtype=torch.uint8, device=dev) if fp8 else \
            torch.zeros((used, 64, 1, 576), dtype=torch.bfloat16, device=dev)
        keys, scales = torch.zeros((used, 576), dtype=torch.int8, device=dev), torch.zeros((used,), device=dev)
        (mla.mla_cache_write_fp8 if fp8 else mla.mla_cache_write)(xd[:, :512], xd[:, 512:], cache, tb, zero, cu)
        (mla.mla_update_page_keys_fp8 if fp8 else mla.mla_update_page_keys)(cache, tb, sl, keys, scales)
        check(dev, q.cpu(), cache.cpu(), table, lens, keys.cpu(), scales.cpu(), 5)
        o, lse, pages = decode(dev, q, cache, tb, lens, keys, scales, 12)
        md, ns = mla.mla_get_metadata(sl, 128, 1)
        o2, lse2 = (mla.mla_decode_kvcache_fp8 if fp8 else mla.mla_decode_kvcache)(q, cache, tb, sl, 512, md, ns)
        if fp8:  # two kernels, each off by at most the bound of assert_attention
            assert float((lse - lse2).abs().max()) <= 4e-3
        else:    # the same kernel on the same pages
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert pages[2, 0].tolist() == [0] + [-1] * 11
        assert mla.mla_device_status() == 0


def test_bad_lengths_and_blocks_are_reported(dev):
    lens = [64 * 6, 64 * 5]
    q, cache, table, keys, scales = make(lens, 1, 16)
    bad = table.clone()
    bad[1, 2] = keys.shape[0]
    o, _, _ = decode(dev, q, cache, bad, lens, keys, scales, 3)
    ref = reference(q, cache, table, lens, keys, scales, 3, 1, 1, False, 576 ** -0.5)
    assert mla.mla_device_status() == _lib.MLA_DEVERR_BLOCK_ID
    assert float((o[0].double().cpu() - ref[0][0]).abs().max()) < 1e-2
    decode(dev, q, cache, table, [64 * 6, -4], keys, scales, 3)
    assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
    decode(dev, q, cache, table, [64 * 6, 64 * table.shape[1] + 1], keys, scales, 3)
    assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN


def test_two_streams_and_a_graph(dev):
    """Calls that overlap on two streams, each with its own workspace, and a captured call with new inputs."""
    lens = [64 * 30 + 9, 64 * 50]
    sets = [make(lens, 2, 16, seed=s) for s in (1, 2)]
    want = [reference(q, c, t, lens, k, s, 6, 1, 1, True, 576 ** -0.5) for q, c, t, k, s in sets]
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    on = [tuple(t.to(dev) for t in s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(dev), torch.cuda.Stream(dev)], [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                q, c, t, k, s = on[i]
                got[i] = mla.mla_decode_kvcache_blocks(q, c, t, sl, k, s, 6, 512, causal=True)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][2].cpu(), want[i][3])
        R.assert_attention(got[i][0], got[i][1], *want[i][:3], False)
    bufs = [t.clone() for t in on[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mla.mla_decode_kvcache_blocks(bufs[0], bufs[1], bufs[2], sl, bufs[3], bufs[4], 6, 512, causal=True)
    for i in (1, 0):
        for dst, src in zip(bufs, on[i]):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[2].cpu(), want[i][3])
        R.assert_attention(out[0], out[1], *want[i][:3], False)
    assert mla.mla_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_far_into_a_large_pool(dev, fp8):
    """Pages whose offsets pass 2^32, and their keys, give the results of the same ones at the pool's start."""
    lens = [900, 300]
    q, cache, table, keys, scales = make(lens, 2, 48, 576, fp8, seed=21)
    want = decode(dev, q, cache, table, lens, keys, scales, 4)
    n = cache.shape[0]
    nblk = 2 ** 32 // (64 * 576) + 64
    pool = torch.empty((nblk, *cache.shape[1:]), dtype=cache.dtype, device=dev)
    pool[-n:] = cache.to(dev)
    far_keys = torch.empty((nblk, 576), dtype=torch.int8, device=dev)
    far_scales = torch.empty((nblk,), device=dev)
    far_keys[-n:], far_scales[-n:] = keys.to(dev), scales.to(dev)
    got = decode(dev, q, pool, table + (nblk - n), lens, far_keys, far_scales, 4)
    assert mla.mla_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_workspace_and_outputs_of_the_caller(dev):
    """A workspace full of NaN that a second call of other lengths reuses; outputs that held something else."""
    lens = [900, 300, 64]
    q, cache, table, keys, scales = make(lens, 2, 48, 576, seed=22)
    need = mla.mla_blocks_workspace_bytes(3, 2, 48, 1, 512, table.shape[1], 4, mla.mla_num_sm_parts(1, 1, dev))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=dev)
    out = torch.full((3, 2, 48, 512), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((3, 2, 48), 7.0, device=dev)
    pages = torch.full((3, 2, 4), 7, dtype=torch.int32, device=dev)
    for now in (lens, [0, 70, 64], [500, 1, 3]):
        ref = reference(q, cache, table, now, keys, scales, 4, 1, 1, True, 576 ** -0.5)
        got = decode(dev, q, cache, table, now, keys, scales, 4, causal=True, out=out, lse=lse, pages=pages, workspace=ws)
        assert mla.mla_device_status() == 0 and got[0] is out and got[2] is pages
        assert torch.equal(pages.cpu(), ref[3])
        R.assert_attention(out, lse, *ref[:3], False)
    with pytest.raises(RuntimeError, match="workspace"):
        decode(dev, q, cache, table, lens, keys, scales, 4, workspace=ws[:need - 256])
    with pytest.raises(ValueError, match="too large"):
        decode(dev, q, cache, table, lens, keys, scales, 1 << 26)


@pytest.mark.parametrize("exponent", [-122, -108, -101, -93, 90])
def test_heads_of_every_magnitude(dev, exponent):
    """The heads' codes are the quotients' also where a reciprocal or a remainder would be subnormal."""
    lens = [900, 650]
    q, cache, table, keys, scales = make(lens, 2, 24, 576, seed=23)
    spread = torch.arange(24).view(1, 1, 24, 1) % 8
    q = (q.float() * 2.0 ** exponent * 2.0 ** spread).to(torch.bfloat16)
    ref = reference(q, cache, table, lens, keys, scales, 5, 1, 1, False, 1.0)
    got = decode(dev, q, cache, table, lens, keys, scales, 5, softmax_scale=1.0)
    assert mla.mla_device_status() == 0
    assert torch.equal(got[2].cpu(), ref[3])


def test_calls_from_several_threads_at_once(dev):
    """Threads with a stream each, both formats, small and full tiles: every call gives the bits it gives alone."""
    import threading
    lens = [1500, 300, 576]
    cases = [make(lens, 2, h, 576, fp8, seed=24) for h, fp8 in ((128, False), (128, True), (32, False), (32, True))]
    cases = [[t.to(dev) for t in c] for c in cases]
    run = lambda c: decode(dev, c[0], c[1], c[2], lens, c[3], c[4], 6)
    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream(dev)
        with torch.cuda.stream(stream):
            got = [run(cases[i]) for _ in range(20)]
            stream.synchronize()
            wrong.extend(i for g in got if not all(torch.equal(a, b) for a, b in zip(want[i], g)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and mla.mla_device_status() == 0
