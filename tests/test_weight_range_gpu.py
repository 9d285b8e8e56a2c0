"""The e4m3 decodes where softmax weights span many magnitudes: a heavy key before, behind or among thousands of
light ones that together hold much of the mass, as an attention sink does."""
import numpy as np
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import workloads as W
from tests import reference64 as R

pytestmark = pytest.mark.gpu

HEADS = 32
GAPS = torch.linspace(4.0, 14.0, HEADS)  # nats between levels 0 and 1, head by head


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_status_left():
    mla.mla_device_status()
    yield


def make(levels, seed=0, small=()):
    """(q [1, 2, 32, 576], pages, table) of one sequence whose key j scores about GAPS[h] * levels[j] for head h.

    The last 64 dims hold the level along one direction; the values have a mean, so that keys that are left out
    show.  Rows `small` have values of a sixteenth: small scales, since their levels then lead their rows."""
    g = torch.Generator().manual_seed(seed)
    T = len(levels)
    n = (T + 63) // 64
    way = torch.randint(0, 2, (64,), generator=g) * 2.0 - 1
    rows = torch.zeros((n * 64, 576))
    mean = torch.rand((512,), generator=g) + 0.5
    rows[:T, :512] = (mean + 0.3 * torch.randn((T, 512), generator=g)) * (16.0 if len(small) else 1.0)
    for j in small:
        rows[j, :512] /= 16.0
    rows[:T, 512:] = levels[:, None] * way
    q = torch.zeros((1, 2, HEADS, 576))
    q[..., :512] = 0.003 * torch.randn((1, 2, HEADS, 512), generator=g)
    q[..., 512:] = GAPS[:, None] * 24.0 / 64.0 * way
    table = torch.randperm(n, generator=g).to(torch.int32)
    cache = torch.zeros((n, 64 * 580), dtype=torch.uint8)
    cache[table.long()] = W.pack_e4m3_pages(rows.view(n, 64, 576))
    return q.to(torch.bfloat16), cache, table[None]


def rows_of(cache, table, T, pages=None):
    rows = R.cache_rows(cache)
    pages = range((T + 63) // 64) if pages is None else pages
    return torch.cat([rows[int(table[0, p])][:min(64, T - 64 * p)] for p in pages])


def reference(q, rows):
    """o, lse, the bound of o, and the sum of the weights relative to the largest, of q [h, 576] over rows [t, 576].

    Rounding o to bf16 is off by at most 2^-8 |o|.  A weight times its token's scale, w, becomes an f16 (2^-11) and
    then two parts: e4m3's half step is 2^-4 of the power of two below w, and e5m2's 2^-8 of it for what is left, so
    2^-8 w; a score's fp32 accumulation adds less than 2^-11.  What weights below the range of the parts lose is
    kept below 2^-9 of the sum of all w, whatever their number, and every code is at most max |row| / scale."""
    z = q.double() @ rows.T * 576 ** -0.5
    top = z.amax(1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(1, keepdim=True)
    p = p / total
    o = p @ rows[:, :512]
    bound = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -10) * (p @ rows[:, :512].abs()) \
        + 2.0 ** -9 * (p @ rows.abs().amax(1))[:, None]
    return o, torch.log(total[:, 0]) + top[:, 0], bound, total[:, 0]


def compare(o, lse, ref, what=""):
    d = (o.double().cpu() - ref[0]).abs() / ref[2]
    assert torch.isfinite(o).all() and float(d.max()) <= 1.0, f"{what}: |dO| is {float(d.max()):.2f} times its bound"
    assert float((lse.double().cpu() - ref[1]).abs().max()) <= 2e-3, what


def check_tree(dev, q, cache, table, T, num_parts):
    lens = torch.tensor([T], dtype=torch.int32, device=dev)
    sees = R.ancestors([-1, 0])
    md, ns = mla.mla_get_metadata_tree(lens, 2, HEADS, num_parts=num_parts)
    dq, dc, dt = q.to(dev), cache.to(dev), table.to(dev)
    o, lse = mla.mla_decode_kvcache_tree_fp8(dq, dc, dt, lens, R.mask_words(sees)[None].to(dev), 512, md, ns)
    assert mla.mla_device_status() == 0
    rows = rows_of(cache, table, T)
    refs = [reference(q[0, 0], rows[:T - 1]), reference(q[0, 1], rows)]
    for i, ref in enumerate(refs):
        compare(o[0, i], lse[0, i], ref, f"token {i}")
    # the dense decode of the same rows: its weights are f16, 2^-11 of themselves or 2^-25 where that is more
    md, ns = mla.mla_get_metadata(lens, 2 * HEADS, num_parts=num_parts)
    dense, _ = mla.mla_decode_kvcache_fp8(dq, dc, dt, lens, 512, md, ns, causal=True)
    codes = rows[:, :512].abs() / (rows.abs().amax(1, keepdim=True) / 448)
    for i, ref in enumerate(refs):
        # (a quarter of the bound covers its 2^-11; its o is rounded too)
        room = 1.25 * ref[2] + 2.0 ** -8 * ref[0].abs() + 2.0 ** -25 * codes.sum(0) / ref[3][:, None]
        assert bool(((o[0, i].double() - dense[0, i].double()).abs().cpu() <= room).all())


def check_blocks(dev, q, cache, table, T, topk):
    lens = torch.tensor([T], dtype=torch.int32, device=dev)
    keys = torch.zeros((cache.shape[0], 576), dtype=torch.int8, device=dev)
    scales = torch.zeros((cache.shape[0],), device=dev)
    dc, dt = cache.to(dev), table.to(dev)
    mla.mla_update_page_keys_fp8(dc, dt, lens, keys, scales)
    o, lse, pages = mla.mla_decode_kvcache_blocks_fp8(q[:, :1].contiguous().to(dev), dc, dt, lens, keys, scales, topk, 512)
    assert mla.mla_device_status() == 0
    pick = [p for p in pages[0, 0].tolist() if p >= 0]
    assert len(pick) == min(topk, (T + 63) // 64) and pick[0] == 0 and pick[-1] == (T + 63) // 64 - 1
    compare(o[0, 0], lse[0, 0], reference(q[0, 0], rows_of(cache, table, T, pick)), "blocks")


def light(T, seed=1):
    return 0.03 * torch.randn((T,), generator=torch.Generator().manual_seed(seed))


def heavy_at(T, *at):
    x = light(T)
    x[list(at)] = 1.0
    return x


LEVELS = {
    "first": lambda T: heavy_at(T, 0),
    "first page's last": lambda T: heavy_at(T, 63),
    "middle": lambda T: heavy_at(T, T // 2),
    "last page": lambda T: heavy_at(T, T - 5),
    "both ends": lambda T: heavy_at(T, 3, T - 5),
    "one in each page": lambda T: heavy_at(T, *range(17, T, 64)),
    "pages in turn": lambda T: light(T) + (torch.arange(T) // 64 % 2 == 0).float(),
    "falling": lambda T: light(T) + torch.clamp(1 - torch.arange(T) // 64 / 6, min=0),
    "rising": lambda T: light(T) + torch.clamp(torch.arange(T) // 64 / 6, max=1),
    "wide": lambda T: 0.25 * torch.randn((T,), generator=torch.Generator().manual_seed(9)),
}


@pytest.mark.parametrize("num_parts", [1, 5])
@pytest.mark.parametrize("T", [64, 512, 4100, 16384])
@pytest.mark.parametrize("levels", LEVELS)
def test_trees(dev, levels, T, num_parts):
    check_tree(dev, *make(LEVELS[levels](T)), T, num_parts)


@pytest.mark.parametrize("topk", [24, 200])
@pytest.mark.parametrize("T", [512, 4100, 12800])
@pytest.mark.parametrize("levels", LEVELS)
def test_selected_pages(dev, levels, T, topk):
    check_blocks(dev, *make(LEVELS[levels](T)), T, topk)


@pytest.mark.parametrize("num_parts", [1, 5])
@pytest.mark.parametrize("at", [0, 2000])
def test_a_heavy_key_of_a_small_scale(dev, at, num_parts):
    """Its weight times its scale is far below what the page's largest scale lets expect."""
    T = 4096
    check_tree(dev, *make(heavy_at(T, at), small=(at,)), T, num_parts)
    check_blocks(dev, *make(heavy_at(T, at), small=(at,)), T, 64)


def test_random_scores_of_many_spreads(dev):
    """Heads whose scores spread from 0.1 to 6 nats over the same N(0, 1) rows, many sequences of odd lengths."""
    g = torch.Generator().manual_seed(4)
    lens = [1, 63, 65, 200, 1000, 3001, 8000]
    table, used = R.random_table(g, lens)
    cache = R.random_cache(g, used, 576, True)
    q = torch.randn((len(lens), 1, HEADS, 576), generator=g) * torch.tensor(
        np.geomspace(0.1, 6.0, HEADS), dtype=torch.float32)[:, None]
    q = q.to(torch.bfloat16)
    o, lse = mla.mla_decode_kvcache_tree_fp8(
        q.to(dev), cache.to(dev), table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
        torch.ones((len(lens), 1, 1), dtype=torch.int32, device=dev), 512)
    assert mla.mla_device_status() == 0
    for b, T in enumerate(lens):
        compare(o[b, 0], lse[b, 0], reference(q[b, 0], rows_of(cache, table[b:b + 1], T)), f"{T} keys")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30, 255.0])
@pytest.mark.parametrize("h", [16, 128])
def test_the_scale_of_a_node_that_nothing_sees(dev, bad, h):
    """It is neither used nor reported; with 128 heads (one token per tile) one that token 6 sees is reported."""
    from mla_decode_attention_latent_gb300 import _lib
    g = torch.Generator().manual_seed(6)
    lens, s_q = [200, 70], 10
    table, used = R.random_table(g, lens)
    cache = R.random_cache(g, used, 576, True)
    q = torch.randn((2, s_q, h, 576), generator=g).to(torch.bfloat16)
    sees = R.ancestors([-1, 0, 0, 1, 2, 3, 0, 1, 1, 0])
    sees[:, 4] = False
    mask = torch.stack([R.mask_words(sees)] * 2).to(dev)
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)

    def decode():
        o, lse = mla.mla_decode_kvcache_tree_fp8(q.to(dev), cache.to(dev), table.to(dev), sl, mask, 512)
        return o, lse, mla.mla_device_status()

    def spoil(node):
        for i, T in enumerate(lens):
            blk, off = R.place(table, i, T - s_q + node)
            cache[blk, 64 * 576 + 4 * off:64 * 576 + 4 * off + 4] = torch.tensor([bad]).view(torch.uint8)
    want = decode()
    spoil(4)
    got = decode()
    assert want[2] == got[2] == 0
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    spoil(6)
    assert decode()[2] == _lib.MLA_DEVERR_SCALE


@pytest.mark.parametrize("s_q,h,lens,num_parts", [
    (1, 16, [1, 64, 65], None), (8, 16, [500, 8, 71], None), (7, 30, [64, 130, 9], 3), (33, 4, [33, 100, 128], None),
    (5, 128, [70, 200], 5), (3, 160, [65, 700, 129], None), (66, 8, [400, 75, 66, 129], 7), (1, 100, [3000, 5000], None)])
def test_trees_of_many_shapes(dev, s_q, h, lens, num_parts):
    """N(0, 1) rows and random trees under the bound above, which does not grow with the number of keys."""
    from tests import test_tree_gpu as trees
    q, cache, table, sees = trees.make(lens, s_q, h, 576, True, seed=s_q)
    o, lse = trees.decode(dev, q, cache, table, lens, sees, num_parts=num_parts)
    assert mla.mla_device_status() == 0
    for b, T in enumerate(lens):
        rows = rows_of(cache, table[b:b + 1], T)
        for i in range(s_q):
            see = [t for t in range(T) if t < T - s_q or sees[b][i, t - (T - s_q)]]
            compare(o[b, i], lse[b, i], reference(q[b, i], rows[see]), f"sequence {b} token {i}")


@pytest.mark.parametrize("s_q,h,lens,topk,causal", [
    (1, 16, [1000, 1, 64, 65, 700], 5, False), (3, 32, [400, 66, 130, 321], 4, True), (1, 160, [900, 64], 8, False),
    (4, 128, [1500, 300, 576], 6, True)])
def test_selected_pages_of_many_shapes(dev, s_q, h, lens, topk, causal):
    from tests import test_blocks_gpu as blocks
    q, cache, table, keys, scales = blocks.make(lens, s_q, h, 576, True, seed=h)
    o, lse, pages = blocks.decode(dev, q, cache, table, lens, keys, scales, topk, causal=causal)
    assert mla.mla_device_status() == 0
    for b, T in enumerate(lens):
        for i in range(s_q):
            n = R.token_len(T, s_q, i, causal)
            pick = [p for p in pages[b, i].tolist() if p >= 0]
            compare(o[b, i], lse[b, i], reference(q[b, i], rows_of(cache, table[b:b + 1], n, pick)), f"{b} {i}")


@pytest.mark.parametrize("softmax_scale", [576 ** -0.5, -576 ** -0.5, 0.0])
def test_scales_of_both_signs(dev, softmax_scale):
    """Rows may be held as negative scales times negated codes, and the softmax scale may have any sign."""
    T = 3000
    q, cache, table = make(heavy_at(T, 0))
    want_rows = rows_of(cache, table, T)
    turned = torch.rand((cache.shape[0], 64), generator=torch.Generator().manual_seed(3)) < 0.5
    codes, scales = cache[:, :64 * 576].view(-1, 64, 576), cache[:, 64 * 576:].view(torch.float32)
    codes[turned] ^= 0x80
    scales[turned] *= -1
    rows = rows_of(cache, table, T)
    assert torch.equal(rows, want_rows)
    lens = torch.tensor([T], dtype=torch.int32, device=dev)
    o, lse = mla.mla_decode_kvcache_tree_fp8(q.to(dev), cache.to(dev), table.to(dev), lens,
                                             R.mask_words(R.ancestors([-1, 0]))[None].to(dev), 512,
                                             softmax_scale=softmax_scale)
    assert mla.mla_device_status() == 0
    for i, n in ((0, T - 1), (1, T)):
        compare(o[0, i], lse[0, i], reference(q[0, i].double() * (softmax_scale * 24), rows[:n]), f"token {i}")


def test_a_long_sequence_behind_a_sink(dev):
    T = 65536 + 77
    check_tree(dev, *make(heavy_at(T, 0)), T, 76)
    check_blocks(dev, *make(heavy_at(T, 0)), T, 512)
