"""Decode of draft trees against 64 bits."""
import numpy as np
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


def random_parents(rng, s):
    return [int(rng.integers(max(-1, i - 6), i)) if i else -1 for i in range(s)]


def make(lens, s_q, h, d=576, fp8=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    table, used = R.random_table(g, lens, extra=1)
    cache = R.random_cache(g, used, d, fp8)
    q = torch.randn((len(lens), s_q, h, d), generator=g).to(torch.bfloat16)
    sees = np.stack([R.ancestors(random_parents(rng, s_q)) for _ in lens])
    return q, cache, table, sees


def words(sees):
    return torch.stack([R.mask_words(s) for s in sees])


def reference(q, cache, table, lens, sees, nodes, scale):
    b, s_q, h, d = q.shape
    rows = R.cache_rows(cache)
    o = torch.zeros((b, s_q, h, 512), dtype=torch.float64)
    a, lse = o.clone(), torch.full((b, s_q, h), -float("inf"), dtype=torch.float64)
    for i in range(b):
        T, n = lens[i], nodes[i]
        flat = torch.cat([rows[int(table[i, p])] for p in range((T + 63) // 64)] + [torch.zeros((0, d), dtype=torch.float64)])[:T]
        for j in range(n):
            see = [p for p in range(T) if p < T - n or sees[i][j, p - (T - n)]]
            o[i, j], lse[i, j], a[i, j] = R.attend(q[i, j], flat[see], scale, cache.dtype != torch.bfloat16)
    return o, lse, a


def decode(dev, q, cache, table, lens, sees, nodes=None, num_parts=None, **k):
    call = mla.mla_decode_kvcache_tree if cache.dtype == torch.bfloat16 else mla.mla_decode_kvcache_tree_fp8
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    if num_parts:
        k["tile_scheduler_metadata"], k["num_splits"] = mla.mla_get_metadata_tree(
            sl, q.shape[1], q.shape[2], None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device=dev),
            num_parts=num_parts)
    return call(q.to(dev), cache.to(dev), table.to(dev), sl, words(sees).to(dev), 512,
                tree_lens=None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device=dev), **k)


def check(dev, q, cache, table, lens, sees, nodes=None, **k):
    ref = reference(q, cache, table, lens, sees, nodes or [q.shape[1]] * len(lens), q.shape[3] ** -0.5)
    o, lse = decode(dev, q, cache, table, lens, sees, nodes, **k)
    assert mla.mla_device_status() == 0
    R.assert_attention(o, lse, *ref, cache.dtype != torch.bfloat16)
    return o, lse


FORMATS = [(576, False), (512, False), (576, True)]


@pytest.mark.parametrize("d,fp8", FORMATS)
@pytest.mark.parametrize("s_q,h,lens", [
    (1, 16, [1, 64, 65]), (8, 16, [500, 8, 71]), (7, 30, [64, 130, 9]), (33, 4, [33, 100, 128]), (5, 128, [70, 200]),
    (65, 16, [65, 700, 129]), (200, 1, [230, 200])])
def test_trees(dev, d, fp8, s_q, h, lens):
    q, cache, table, sees = make(lens, s_q, h, d, fp8)
    check(dev, q, cache, table, lens, sees)


@pytest.mark.parametrize("d,fp8", FORMATS)
@pytest.mark.parametrize("num_parts", [1, 3, 7])
def test_split_trees(dev, d, fp8, num_parts):
    """Sequences cut between parts, also inside the pages that hold nodes."""
    lens = [400, 75, 66, 129]
    q, cache, table, sees = make(lens, 66, 8, d, fp8, seed=3)
    check(dev, q, cache, table, lens, sees, num_parts=num_parts)


@pytest.mark.parametrize("d,fp8", FORMATS)
def test_trees_of_several_sizes(dev, d, fp8):
    """A padded batch: rows behind a tree see nothing; a sequence without nodes, and one without anything."""
    lens, nodes = [300, 64, 12, 100, 0], [13, 5, 12, 0, 0]
    q, cache, table, sees = make(lens, 13, 32, d, fp8)
    o, lse = check(dev, q, cache, table, lens, sees, nodes)
    assert not o[3].any() and bool(torch.isneginf(lse[3:]).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_sequence_shorter_than_its_tree(dev, fp8):
    """Nodes that would lie before the sequence do not exist; the others keep their bits."""
    lens = [5, 70]
    q, cache, table, sees = make(lens, 80, 2, 576, fp8)
    rows = R.cache_rows(cache)
    o, lse = decode(dev, q, cache, table, lens, sees)
    assert mla.mla_device_status() == 0
    for i, T in enumerate(lens):
        flat = torch.cat([rows[int(table[i, p])] for p in range((T + 63) // 64)])[:T]
        for j in range(80):
            see = [p for p in range(T) if sees[i][j, p - (T - 80)]]
            r = R.attend(q[i, j], flat[see], 576 ** -0.5, fp8)
            R.assert_attention(o[i, j], lse[i, j], *r, fp8, f"{i} {j}")


@pytest.mark.parametrize("fp8", [False, True])
def test_any_mask(dev, fp8):
    """Random bits, rows that see no node, and with no prefix a row that sees nothing."""
    lens = [40, 150, 90]
    q, cache, table, _ = make(lens, 40, 16, 576, fp8)
    rng = np.random.default_rng(1)
    sees = rng.random((3, 40, 40)) < 0.3
    sees[0, 5] = sees[1, 7] = False
    o, lse = check(dev, q, cache, table, lens, sees)
    assert not o[0, 5].any() and bool(torch.isneginf(lse[0, 5]).all())


@pytest.mark.parametrize("d", [576, 512])
@pytest.mark.parametrize("s_q,h", [(8, 128), (40, 16)])
def test_a_chain_is_the_causal_decode(dev, d, s_q, h):
    """Bit for bit, where no sequence is cut between parts."""
    lens = [300, 128, 64, 41]
    q, cache, table, _ = make(lens, s_q, h, d)
    sees = np.stack([np.tril(np.ones((s_q, s_q), bool))] * 4)
    o, lse = decode(dev, q, cache, table, lens, sees, num_parts=1)
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    md, ns = mla.mla_get_metadata(sl, s_q * h, 1, num_parts=1)
    o2, lse2 = mla.mla_decode_kvcache(q.to(dev), cache.to(dev), table.to(dev), sl, 512, md, ns, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and mla.mla_device_status() == 0


@pytest.mark.parametrize("d,fp8", FORMATS)
@pytest.mark.parametrize("h", [16, 128])
def test_rows_that_nothing_sees_may_hold_anything(dev, d, fp8, h):
    """NaN and infinities past the end, in unused pages, and in a node that no token sees; with 128 heads (one
    token per tile) also in a node that another token sees."""
    lens = [200, 70]
    q, cache, table, sees = make(lens, 10, h, d, fp8)
    sees[:, :, 4] = False
    if h == 128:
        sees[:, :, 6] = False
        sees[:, 6, 6] = True

    def spoil(blk, off, v):
        if fp8:
            cache[blk, off * d:(off + 1) * d] = 0x7f
            if off >= 8:  # past the end: the scale too
                cache[blk, 64 * d + 4 * off:64 * d + 4 * off + 4] = torch.tensor([v]).view(torch.uint8)
        else:
            cache[blk, off, 0] = v
    ref_cache = cache.clone()
    for i, T in enumerate(lens):
        for p in range(T, 64 * ((T + 63) // 64)):
            spoil(*R.place(table, i, p), float("nan"))
        for node in [4] + ([6] if h == 128 else []):
            blk, off = R.place(table, i, T - 10 + node)
            if fp8:
                cache[blk, off * d:(off + 1) * d] = 0x7f
            else:
                cache[blk, off, 0] = float("nan") if node == 4 else float("inf")
    ref = reference(q, ref_cache, table, lens, sees, [10, 10], d ** -0.5)
    o, lse = decode(dev, q, cache, table, lens, sees)
    assert mla.mla_device_status() == 0
    rows = [i for i in range(10) if h < 128 or i != 6]
    R.assert_attention(o[:, rows], lse[:, rows], *(t[:, rows] for t in ref), fp8)


def test_bad_tree_lengths_are_reported(dev):
    lens = [100, 100]
    q, cache, table, sees = make(lens, 6, 16)
    for bad, n in ((-1, 0), (7, 6)):
        ref = reference(q, cache, table, lens, sees, [6, n], 576 ** -0.5)
        o, lse = decode(dev, q, cache, table, lens, sees, [6, bad])
        assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
        R.assert_attention(o, lse, *ref, False)


@pytest.mark.parametrize("s_q", [1, 2, 31, 32, 33, 64, 100, 513])
def test_tree_mask(dev, s_q):
    rng = np.random.default_rng(s_q)
    parents = [random_parents(rng, s_q) for _ in range(3)]
    parents[1] = [-1] * s_q
    parents[2] = list(range(-1, s_q - 1))
    got = mla.mla_tree_mask(torch.tensor(parents, dtype=torch.int32, device=dev))
    assert torch.equal(got.cpu(), words([R.ancestors(p) for p in parents])) and mla.mla_device_status() == 0


def test_tree_mask_reports_bad_parents(dev):
    for bad in (-2, 3, 2 ** 31 - 1, -2 ** 31):
        got = mla.mla_tree_mask(torch.tensor([[-1, 0, 1, bad, 3]], dtype=torch.int32, device=dev))
        assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
        assert torch.equal(got.cpu()[0], R.mask_words(R.ancestors([-1, 0, 1, -1, 3])))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_step_of_speculative_decoding(dev, fp8):
    """Drafts written, masks from parents, tree decode, the accepted path committed by another write, page keys
    updated, decode over selected pages, rows read back; the calls follow one another on one stream."""
    g = torch.Generator().manual_seed(2)
    past, s_q, h = [64 * 8 + 3, 127], 6, 128
    lens = [t + s_q for t in past]
    table, used = R.random_table(g, lens)
    parents = [[-1, 0, 0, 1, 2, 4], [-1, -1, 1, 2, 2, 0]]
    ref = R.random_cache(g, used, 576, fp8)
    draft = torch.randn((2 * s_q, 576), generator=g).to(torch.bfloat16)
    q = torch.randn((2, s_q, h, 576), generator=g).to(torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cache, tb, x, qd = ref.to(dev), table.to(dev), draft.to(dev), q.to(dev)
    write = mla.mla_cache_write_fp8 if fp8 else mla.mla_cache_write
    write(x[:, :512], x[:, 512:], cache, tb, i32(past))
    mask = mla.mla_tree_mask(i32(parents))
    tree = mla.mla_decode_kvcache_tree_fp8 if fp8 else mla.mla_decode_kvcache_tree
    o, lse = tree(qd, cache, tb, i32(lens), mask, 512)
    sees = [R.ancestors(p) for p in parents]
    with_drafts = cache.cpu()
    R.assert_attention(o, lse, *reference(q, with_drafts, table, lens, sees, [s_q] * 2, 576 ** -0.5), fp8)
    # paths 0 -> 2 -> 4 and 1 -> 2 are accepted: their rows become the sequences' next ones
    kept = [[0, 2, 4], [1, 2]]
    rows = x[torch.tensor([k + s_q * b for b, ks in enumerate(kept) for k in ks], device=dev)]
    write(rows[:, :512], rows[:, 512:], cache, tb, i32(past), cu_rows=i32([0, 3, 5]))
    now = [past[0] + 3, past[1] + 2]
    keys, scales = torch.zeros((used, 576), dtype=torch.int8, device=dev), torch.zeros((used,), device=dev)
    update = mla.mla_update_page_keys_fp8 if fp8 else mla.mla_update_page_keys
    update(cache, tb, i32(now), keys, scales)
    blocks = mla.mla_decode_kvcache_blocks_fp8 if fp8 else mla.mla_decode_kvcache_blocks
    o, lse, pages = blocks(qd[:, :1].contiguous(), cache, tb, i32(now), keys, scales, 4, 512)
    lat, rope = (mla.mla_cache_read_fp8 if fp8 else mla.mla_cache_read)(cache, tb, i32(past), 5, cu_rows=i32([0, 3, 5]))
    assert mla.mla_device_status() == 0
    from tests.test_blocks_gpu import reference as blocks_reference
    ro, rl, ra, rp = blocks_reference(q[:, :1], cache.cpu(), table, now, keys.cpu(), scales.cpu(), 4, 1, 1, False, 576 ** -0.5)
    assert torch.equal(pages.cpu(), rp)
    R.assert_attention(o, lse, ro, rl, ra, fp8)
    r64 = R.cache_rows(cache.cpu())
    got, r = torch.cat([lat, rope], 1).cpu(), 0
    for b, ks in enumerate(kept):
        for i in range(len(ks)):
            assert torch.equal(got[r], R.f32(r64[R.place(table, b, past[b] + i)]).to(torch.bfloat16))
            if not fp8:
                assert torch.equal(got[r], draft[ks[i] + s_q * b])
            r += 1


def test_in_a_graph_and_on_another_stream(dev):
    lens = [300, 90]
    q, cache, table, sees = make(lens, 9, 16)
    q2, cache2, table2, sees2 = make(lens, 9, 16, seed=8)
    want = [reference(*v, [9, 9], 576 ** -0.5) for v in ((q, cache, table, lens, sees), (q2, cache2, table2, lens, sees2))]
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    ins = [(a.to(dev), b.to(dev), c.to(dev), words(s).to(dev)) for a, b, c, s in ((q, cache, table, sees), (q2, cache2, table2, sees2))]
    bufs = [t.clone() for t in ins[0]]
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    with torch.cuda.stream(s):
        o, lse = mla.mla_decode_kvcache_tree(bufs[0], bufs[1], bufs[2], sl, bufs[3], 512)
    s.synchronize()
    R.assert_attention(o, lse, *want[0], False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = mla.mla_decode_kvcache_tree(bufs[0], bufs[1], bufs[2], sl, bufs[3], 512)
    for i in (1, 0):
        for dst, src in zip(bufs, ins[i]):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        R.assert_attention(o, lse, *want[i], False)
    assert mla.mla_device_status() == 0


def test_partition_over_row_tiles(dev):
    """mla_get_metadata_tree is the decode's partition of the tiles' lengths, bit for bit."""
    import oracle
    rng = np.random.default_rng(6)
    for b, s_q, h, parts in ((1, 1, 16, 76), (3, 13, 64, 76), (16, 32, 128, 76), (5, 33, 100, 3), (300, 9, 128, 11)):
        lens = rng.integers(0, 3000, b)
        nodes = rng.integers(0, s_q + 1, b)
        tiles = -(-s_q * h // 128)
        for given in (None, nodes):
            flat = [0 if given is not None and t * 128 // h >= given[i] else lens[i] for i in range(b) for t in range(tiles)]
            want = oracle.schedule(np.array(flat), parts)
            got = mla.mla_get_metadata_tree(torch.tensor(lens, dtype=torch.int32, device=dev), s_q, h,
                                            None if given is None else torch.tensor(nodes, dtype=torch.int32, device=dev),
                                            num_parts=parts)
            assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])


@pytest.mark.parametrize("d,fp8,max_exp", [(576, False, 40.0), (512, False, 40.0), (576, True, 10.0)])
@pytest.mark.parametrize("jump,starts", [(11.0, [0, 4, 9, 14]), (5.0, [0, 2, 4, 6, 8, 10, 12, 14]), (7.5, [0, 1, 2, 3, 11, 12, 13])])
@pytest.mark.parametrize("num_parts", [1, 3])
def test_scores_that_climb(dev, d, fp8, max_exp, jump, starts, num_parts):
    """The running maximum rises again and again, by more and by less than the lazy rescale lets pass, and what
    older rows lose in weight their values make up for."""
    from mla_decode_attention_latent_gb300 import workloads as W
    lens, s_q, h = [1000, 700], 3, 64
    c = W.Case("climb", batch=2, s_q=s_q, h_q=h, seqlens=tuple(lens), seed=300, d=d, fp8=fp8)
    x = W.staircase(W.make_inputs(c, "cpu"), starts, jump_log2=jump, max_exp=max_exp)
    sees = np.stack([R.ancestors([-1, 0, 0])] * 2)
    check(dev, x.q, x.kcache, x.block_table, lens, sees, num_parts=num_parts)


@pytest.mark.parametrize("num_parts", [1, 3])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_scales_of_many_sizes(dev, order, num_parts):
    """e4m3 rows whose scales span 2^20, rising, falling and mixed along the sequence, with nearly even weights: the
    range that the weights take in the fp8 product follows the largest, and small rows must not disturb it."""
    from mla_decode_attention_latent_gb300 import workloads as W
    g = torch.Generator().manual_seed(7)
    lens, s_q, h = [900, 500], 2, 64
    table, used = R.random_table(g, lens)
    rows = torch.randn((used, 64, 576), generator=g)
    for b, T in enumerate(lens):
        e = torch.linspace(-14, 6, T) if order == "up" else torch.linspace(6, -14, T) if order == "down" else \
            torch.rand((T,), generator=g) * 20 - 14
        for t in range(T):
            rows[R.place(table, b, t)] *= 2.0 ** float(e[t])
    q = (torch.randn((2, s_q, h, 576), generator=g) * 2.0 ** -9).to(torch.bfloat16)
    cache = W.pack_e4m3_pages(rows)
    check(dev, q, cache, table, lens, np.stack([R.ancestors([-1, 0])] * 2), num_parts=num_parts)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("num_parts", [1, 5])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(dev, fp8, bad, num_parts):
    """The heads of a token share a tile, and their maxima one decision: the other rows keep their bits."""
    lens = [700, 90]
    q, cache, table, sees = make(lens, 4, 24, 576, fp8, seed=11)
    o, lse = decode(dev, q, cache, table, lens, sees, num_parts=num_parts)
    spoilt = q.clone()
    spoilt[0, 1, 5, 100] = bad
    o2, lse2 = decode(dev, spoilt, cache, table, lens, sees, num_parts=num_parts)
    assert mla.mla_device_status() == 0
    keep = torch.ones(o.shape[:3], dtype=torch.bool)
    keep[0, 1, 5] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert bool(torch.isnan(o2[0, 1, 5]).all()) and bool(torch.isnan(lse2[0, 1, 5]))


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_far_into_a_large_pool(dev, fp8):
    """Pages whose byte and element offsets pass 2^32 give the results of the same pages at the pool's start."""
    lens, s_q, h = [300, 130], 5, 32
    q, cache, table, sees = make(lens, s_q, h, 576, fp8, seed=12)
    want = decode(dev, q, cache, table, lens, sees)
    n = cache.shape[0]
    nblk = 2 ** 32 // (64 * 576) + 64
    pool = torch.empty((nblk, *cache.shape[1:]), dtype=cache.dtype, device=dev)
    pool[-n:] = cache.to(dev)
    got = decode(dev, q, pool, table + (nblk - n), lens, sees)
    assert mla.mla_device_status() == 0
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_workspace_and_outputs_of_the_caller(dev, fp8):
    """A workspace full of NaN, reused by a second call of other lengths; outputs that held something else."""
    lens, s_q, h = [1000, 64, 333], 6, 40
    q, cache, table, sees = make(lens, s_q, h, 576, fp8, seed=13)
    need = mla.mla_tree_workspace_bytes(3, s_q, h, 1, 512, mla.mla_num_sm_parts(1, 1, dev))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=dev)
    out = torch.full((3, s_q, h, 512), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((3, s_q, h), 7.0, device=dev)
    check(dev, q, cache, table, lens, sees, out=out, lse=lse, workspace=ws)
    short = [70, 6, 65]
    o, l2 = check(dev, q, cache, table, short, sees, out=out, lse=lse, workspace=ws)
    assert o is out and l2 is lse
    with pytest.raises(RuntimeError, match="workspace"):
        decode(dev, q, cache, table, lens, sees, workspace=ws[:need - 256])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("num_parts", [1, 5])
def test_a_visible_key_that_is_not_finite_shows(dev, fp8, num_parts):
    """In one part of a cut sequence, or in the only one: o and lse of the tokens that see it are NaN."""
    lens, s_q, h = [700, 90], 1, 128
    q, cache, table, sees = make(lens, s_q, h, 576, fp8, seed=14)
    want = decode(dev, q, cache, table, lens, sees, num_parts=num_parts)
    blk, off = R.place(table, 0, 130)
    if fp8:
        cache[blk, off * 576:(off + 1) * 576] = 0x7f
    else:
        cache[blk, off] = float("nan")
    o, lse = decode(dev, q, cache, table, lens, sees, num_parts=num_parts)
    assert mla.mla_device_status() == 0
    assert bool(torch.isnan(o[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert torch.equal(o[1], want[0][1]) and torch.equal(lse[1], want[1][1])
