"""Prompt attention against the formula in 64 bits.

Bounds.  A score is an fp32 sum of at most 192 exact products, off by at most 192 2^-24 of the sum of their magnitudes
(2^-16 is asked, which leaves room for the scaled difference to the maximum); call that e, in units of the scaled
score.  A weight is off by e and by half a bf16 step, 2^-8 of itself, where it multiplies a value (its sum takes it in
fp32), and the sum over values adds fp32 roundings, 2^-23 for each of at most 2^11 products of 16 keys: 2^-12.  So o is
within (2^-8 + 2^-12 + 2 e) sum p |v| of the exact sum, then rounded (2^-8 of o); lse within e + 2^-18 + 2^-22 |lse|.
Where the keys were cut, the parts' joining adds a few roundings of 2^-22.
"""
import math
import threading

import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_status_left():
    mla.mla_device_status()
    yield


def i32(v, dev):
    return torch.tensor(list(v), dtype=torch.int32, device=dev)


def cu_of(lens, dev):
    return torch.nn.functional.pad(torch.tensor(lens).cumsum(0), (1, 0)).to(torch.int32).to(dev)


def make(dev, lq, lk, hq, hkv, rope, seed=0, pad=0, gain=2.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    nq, nk = sum(lq) + pad, sum(lk) + pad
    q = (gain * torch.randn((nq, hq, 192 if rope else 128), generator=g, device=dev)).to(torch.bfloat16)
    up = torch.randn((nk, hkv, 256), generator=g, device=dev).to(torch.bfloat16)
    kr = torch.randn((nk, 64), generator=g, device=dev).to(torch.bfloat16) if rope else None
    return q, up[..., :128], up[..., 128:], kr


def check(out, lse, q, k, v, kr, lq, lk, causal, scale=None, heads=None):
    hq, hkv = q.shape[1], k.shape[1]
    scale = scale or q.shape[-1] ** -0.5
    a = c = 0
    for n, m in zip(lq, lk):
        seen = torch.ones((n, m), dtype=torch.bool, device=q.device)
        if causal:
            seen = seen.tril(m - n)
        for h in heads or range(hq):
            kk = k[c:c + m, h // (hq // hkv)].double()
            if kr is not None:
                kk = torch.cat([kk, kr[c:c + m].double()], 1)
            x = q[a:a + n, h].double()
            vv = v[c:c + m, h // (hq // hkv)].double()
            z = (x @ kk.T * scale).masked_fill(~seen, -math.inf)
            e = 2.0 ** -16 * ((x.abs() @ kk.abs().T) * scale).masked_fill(~seen, 0).amax(1) if m else torch.zeros((n,), device=q.device)
            want = torch.logsumexp(z, 1) if m else torch.full((n,), -math.inf, dtype=torch.float64, device=q.device)
            p = torch.exp(z - torch.where(want > -math.inf, want, 0)[:, None])
            o, spread = p @ vv, p @ vv.abs()
            got, got_lse = out[a:a + n, h].double(), lse[a:a + n, h].double()
            off = (got - o).abs() <= (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -20 + 2 * e)[:, None] * spread + 2.0 ** -8 * o.abs() * 1.01
            good = bool(off.all())
            assert good, (n, m, h, float((got - o).abs().max()))
            none = want == -math.inf
            empty = bool((got_lse[none] == -math.inf).all()) and bool((got[none] == 0).all())
            assert empty
            near = (got_lse - want).abs() <= e + 2.0 ** -18 + 2.0 ** -22 * want.abs()
            good = bool(near[~none].all())
            assert good, (n, m, h, float((got_lse - want)[~none].abs().max()))
        a, c = a + n, c + m


CASES = [
    # lq, lk, hq, hkv
    ([1], [1], 1, 1), ([128], [128], 2, 2), ([256], [256], 2, 1), ([257], [257], 2, 2), ([333], [333], 16, 16),
    ([5, 0, 130, 1, 77], [5, 0, 130, 1, 77], 4, 4),                       # packed, an empty sequence between
    ([3, 64, 200], [500, 64, 1030], 4, 2),                                # chunks behind contexts
    ([100, 7, 40], [30, 0, 40], 2, 2),                                    # rows before the first key; no keys at all
    ([129, 300], [129, 300], 8, 2), ([50, 333], [50, 400], 10, 2),        # groups of 4 and 5 (which leaves rows of a tile empty)
    ([9, 40], [90, 40], 16, 1), ([3, 2], [200, 2], 128, 1), ([700], [700], 12, 4),
    ([15, 16, 17, 31, 33], [15, 16, 17, 31, 33], 3, 3),                   # around the 16 keys of a product
    ([127, 129, 255], [127, 129, 255], 2, 2), ([1, 2, 3], [1025, 4000, 129], 6, 3),
]


@pytest.mark.parametrize("lq,lk,hq,hkv", CASES)
@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("causal", [True, False])
def test_small(dev, lq, lk, hq, hkv, rope, causal):
    q, k, v, kr = make(dev, lq, lk, hq, hkv, rope, seed=sum(lq) + hq)
    out, lse = mla.mla_prefill(q, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr, causal=causal)
    torch.cuda.synchronize()
    assert mla.mla_device_status() == 0
    check(out, lse, q, k, v, kr, lq, lk, causal)


@pytest.mark.parametrize("lq,lk,hq,hkv", [([2000], [2000], 32, 32), ([1500, 3, 900], [1500, 2003, 4000], 32, 8), ([64, 100], [9000, 16384], 16, 16),
                                          ([1], [20000], 8, 8), ([17], [40000], 16, 2), ([4096], [4096], 128, 128), ([300] * 9, [300] * 9, 128, 128)])
@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("causal", [True, False])
def test_large(dev, lq, lk, hq, hkv, rope, causal):
    """More work than SMs, and few rows over many keys (cut blocks)."""
    q, k, v, kr = make(dev, lq, lk, hq, hkv, rope, seed=lq[0])
    out, lse = mla.mla_prefill(q, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr, causal=causal)
    assert mla.mla_device_status() == 0
    check(out, lse, q, k, v, kr, lq, lk, causal, heads=sorted({0, hq // 3, hq // 2 + 1, hq - 1}) if hq > 4 else None)


def test_many_sequences(dev):
    """More sequences than the partition holds at once, most of them short."""
    g = torch.Generator().manual_seed(4)
    lq = torch.randint(0, 9, (2300,), generator=g).tolist()
    lk = [n + int(x) for n, x in zip(lq, torch.randint(0, 20, (2300,), generator=g))]
    q, k, v, kr = make(dev, lq, lk, 2, 2, True)
    out, lse = mla.mla_prefill(q, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr)
    assert mla.mla_device_status() == 0
    check(out, lse, q, k, v, kr, lq, lk, True)


@pytest.mark.parametrize("rope", [True, False])
def test_other_rows_may_hold_anything(dev, rope):
    """Rows between and behind the sequences are NaN and infinite, in queries, keys and values; outputs there stay."""
    lq, lk, pad = [70, 33, 129, 1], [70, 50, 333, 9], 40
    q, k, v, kr = make(dev, lq, lk, 4, 2, rope, pad=pad)
    nq, nk = sum(lq), sum(lk)
    # a hole after every sequence
    at_q, at_k, rows_q, rows_k = [0], [0], [], []
    for n, m in zip(lq, lk):
        rows_q += list(range(at_q[-1], at_q[-1] + n))
        rows_k += list(range(at_k[-1], at_k[-1] + m))
        at_q.append(at_q[-1] + n)
        at_k.append(at_k[-1] + m)
    want, want_lse = mla.mla_prefill(q[:nq], k[:nk], v[:nk], i32(at_q, dev), i32(at_k, dev), k_rope=None if kr is None else kr[:nk])
    for bad in (math.nan, math.inf):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        q2[nq:], k2[nk:], v2[nk:] = bad, bad, bad
        kr2 = None if kr is None else kr.clone()
        if rope:
            kr2[nk:] = bad
        out, lse = torch.full((nq + pad, 4, 128), 5.0, dtype=torch.bfloat16, device=dev), torch.full((nq + pad, 4), 5.0, device=dev)
        mla.mla_prefill(q2, k2, v2, i32(at_q, dev), i32(at_k, dev), k_rope=kr2, out=out, lse=lse)
        assert torch.equal(out[:nq], want) and torch.equal(lse[:nq], want_lse)
        assert (out[nq:] == 5).all() and (lse[nq:] == 5).all()
        # each sequence alone, its neighbours not finite
        for b in range(len(lq)):
            q2, k2, v2 = q.clone(), k.clone(), v.clone()
            mine_q, mine_k = slice(at_q[b], at_q[b + 1]), slice(at_k[b], at_k[b + 1])
            for t, own, other in ((q2, q, mine_q), (k2, k, mine_k), (v2, v, mine_k)):
                t[:] = bad
                t[other] = own[other]
            kr2 = None if kr is None else torch.full_like(kr, bad)
            if rope:
                kr2[mine_k] = kr[mine_k]
            out, lse = mla.mla_prefill(q2, k2, v2, i32(at_q[b:b + 2], dev), i32(at_k[b:b + 2], dev), k_rope=kr2)
            assert torch.equal(out[mine_q], want[mine_q]) and torch.equal(lse[mine_q], want_lse[mine_q])
    assert mla.mla_device_status() == 0


def test_a_query_that_is_not_finite_keeps_to_itself(dev):
    lq, lk = [200], [300]
    q, k, v, kr = make(dev, lq, lk, 2, 2, True)
    want, want_lse = mla.mla_prefill(q, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr)
    q[17, 0, 3], q[150, 1, 190] = math.nan, math.inf
    out, lse = mla.mla_prefill(q, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr)
    good = torch.ones((200, 2), dtype=torch.bool, device=dev)
    good[17, 0] = good[150, 1] = False
    assert torch.equal(out[good], want[good]) and torch.equal(lse[good], want_lse[good])
    assert out[~good].isnan().all() and lse[~good].isnan().all()


def test_maxima_that_grow(dev):
    """Scores that climb by more than 2^8 at chosen steps (O is rescaled), fall, and climb a little (it is not)."""
    n, m = 140, 128 * 9 + 5
    q, k, v, _ = make(dev, [n], [m], 2, 2, False, seed=8, gain=0.5)
    up = torch.zeros((m,), device=dev)
    for at, height in ((130, 9.0), (300, 20.0), (301, -30.0), (600, 60.0), (700, 63.0), (1100, 95.0), (1150, 140.0)):
        up[at:] = height
    q[..., 0] = 128 ** 0.5
    k[..., 0] = up[:, None].to(torch.bfloat16)
    v = (v.float() * torch.exp2(((140.0 - up) / 4).clamp(max=30))[:, None, None]).to(torch.bfloat16)
    for causal in (False, True):
        out, lse = mla.mla_prefill(q, k, v, cu_of([n], dev), cu_of([m], dev), causal=causal)
        check(out, lse, q, k, v, None, [n], [m], causal)


def test_strides_and_scales(dev):
    """Heads outside tokens, keys and values of one projection, one key head, small and large scales."""
    n, m = 150, 210
    q = torch.randn((6, n, 192), device=dev).to(torch.bfloat16).transpose(0, 1)
    up = torch.randn((m, 3, 264), device=dev).to(torch.bfloat16)
    k, v, kr = up[..., :128], up[..., 136:], torch.randn((m, 80), device=dev).to(torch.bfloat16)[:, 8:72]
    for scale in (1e-4, 0.3, 2.0):
        out, lse = mla.mla_prefill(q, k, v, cu_of([n], dev), cu_of([m], dev), k_rope=kr, softmax_scale=scale)
        check(out, lse, q, k, v, kr, [n], [m], True, scale)
    one = up[:, :1]
    out, lse = mla.mla_prefill(q, one[..., :128], one[..., 136:], cu_of([n], dev), cu_of([m], dev), k_rope=kr)
    check(out, lse, q, one[..., :128], one[..., 136:], kr, [n], [m], True)


def test_the_partition_serves_every_layer_and_a_graph(dev):
    lq, lk = [300, 20, 64], [300, 5000, 64]
    cq, ck = cu_of(lq, dev), cu_of(lk, dev)
    layers = [make(dev, lq, lk, 8, 8, True, seed=s) for s in range(3)]
    want = [mla.mla_prefill(q, k, v, cq, ck, k_rope=kr) for q, k, v, kr in layers]
    md = mla.mla_get_metadata_prefill(cq, ck, 384, 5364, 8, 8)
    for (q, k, v, kr), (o, l) in zip(layers, want):
        out, lse = mla.mla_prefill(q, k, v, cq, ck, k_rope=kr, metadata=md)
        assert torch.equal(out, o) and torch.equal(lse, l)
    # captured; replayed on other inputs and other bounds
    q, k, v, kr = (t.clone() for t in layers[0])
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    ws = torch.empty((mla.mla_prefill_workspace_bytes(3, 384, 8, 8),), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_prefill(q, k, v, cq, ck, k_rope=kr, out=out, lse=lse, workspace=ws)
    for i in (1, 2):
        for t, s in zip((q, k, v, kr), layers[i]):
            t.copy_(s)
        graph.replay()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    lq, lk = [10, 350, 24], [4000, 1300, 64]
    cq.copy_(cu_of(lq, dev))
    ck.copy_(cu_of(lk, dev))
    graph.replay()
    check(out, lse, q, k, v, kr, lq, lk, True)
    assert mla.mla_device_status() == 0


def test_the_same_bits_every_time(dev):
    # the last: many items of one length, of which some are cut
    for lq, lk, hq, hkv in (([900, 5, 130], [900, 9000, 2000], 16, 4), ([64] * 37, [5000] * 37, 8, 8)):
        q, k, v, kr = make(dev, lq, lk, hq, hkv, True)
        first = mla.mla_prefill(q, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr)
        for _ in range(5):
            again = mla.mla_prefill(q, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_streams_and_threads(dev):
    """Calls from several threads on streams of their own at once."""
    lq, lk = [200, 40], [200, 3000]
    sets = [make(dev, lq, lk, 8, 8, True, seed=s) for s in range(4)]
    cq, ck = cu_of(lq, dev), cu_of(lk, dev)
    want = [mla.mla_prefill(q, k, v, cq, ck, k_rope=kr) for q, k, v, kr in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            q, k, v, kr = sets[i]
            with torch.cuda.stream(torch.cuda.Stream(dev)) as _:
                for _ in range(10):
                    out, lse = mla.mla_prefill(q, k, v, cq, ck, k_rope=kr)
                    if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])):
                        wrong.append(i)
        except Exception as error:  # pragma: no cover
            wrong.append(error)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_bounds_that_make_no_sense(dev):
    """The sequence is skipped and reported; the others are computed."""
    q, k, v, kr = make(dev, [40, 30], [40, 30], 2, 2, True)
    for cq, ck in (([0, 40, 30], [0, 40, 70]), ([0, 40, 71], [0, 40, 70]), ([0, 40, 70], [0, 40, 71]), ([0, 40, 70], [0, 40, 10])):
        out, lse = torch.full((70, 2, 128), 5.0, dtype=torch.bfloat16, device=dev), torch.full((70, 2), 5.0, device=dev)
        mla.mla_prefill(q, k, v, i32(cq, dev), i32(ck, dev), k_rope=kr, out=out, lse=lse)
        assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
        check(out[:40], lse[:40], q, k, v, kr, [40], [40], True)
        assert (out[40:] == 5).all() and (lse[40:] == 5).all()


def test_no_rows(dev):
    q, k, v, kr = make(dev, [0], [5], 2, 2, True)
    out, lse = mla.mla_prefill(q, k, v, i32([0, 0], dev), i32([0, 5], dev), k_rope=kr)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)
    q, k, v, kr = make(dev, [3], [0], 2, 2, True)
    out, lse = mla.mla_prefill(q, k, v, i32([0, 3], dev), i32([0, 0], dev), k_rope=kr)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert mla.mla_device_status() == 0


def test_rows_beyond_32_bits(dev):
    """Element offsets of queries, keys and outputs pass 2^31."""
    nq, h = 2 ** 31 // (128 * 128) + 300, 128
    q = torch.zeros((nq, h, 128), dtype=torch.bfloat16, device=dev)
    up = torch.zeros((nq, h, 256), dtype=torch.bfloat16, device=dev)
    q[-260:] = torch.randn((260, h, 128), device=dev).to(torch.bfloat16)
    up[-260:] = torch.randn((260, h, 256), device=dev).to(torch.bfloat16)
    out, lse = torch.full((nq, h, 128), 5.0, dtype=torch.bfloat16, device=dev), torch.empty((nq, h), device=dev)
    k, v = up[..., :128], up[..., 128:]
    mla.mla_prefill(q, k, v, i32([nq - 260, nq], dev), i32([nq - 260, nq], dev), out=out, lse=lse)
    check(out[-260:], lse[-260:], q[-260:], k[-260:], v[-260:], None, [260], [260], True, heads=[0, 77, 127])
    assert (out[:-260] == 5).all()
    assert mla.mla_device_status() == 0


@pytest.mark.parametrize("hq,hkv", [(4, 4), (6, 2), (10, 2), (7, 1), (100, 2)])
def test_tiles_with_rows_of_no_query(dev, hq, hkv):
    """Tiles that groups do not fill, or that end inside a sequence, whose other rows are the next sequence's: finite or not."""
    lq, lk = [20, 140, 33, 129, 1, 270], [300, 140, 700, 129, 400, 1500]
    q, k, v, kr = make(dev, lq, lk, hq, hkv, True, seed=hq)
    out, lse = mla.mla_prefill(q, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr)
    check(out, lse, q, k, v, kr, lq, lk, True)
    at = cu_of(lq, dev).tolist()
    for bad in (math.nan, math.inf, 3e38):
        for odd in (0, 1):
            q2 = q.clone()
            for b in range(odd, len(lq), 2):
                q2[at[b]:at[b + 1]] = bad
            o2, l2 = mla.mla_prefill(q2, k, v, cu_of(lq, dev), cu_of(lk, dev), k_rope=kr)
            for b in range(1 - odd, len(lq), 2):
                assert torch.equal(o2[at[b]:at[b + 1]], out[at[b]:at[b + 1]]) and torch.equal(l2[at[b]:at[b + 1]], lse[at[b]:at[b + 1]])
    assert mla.mla_device_status() == 0


def test_weights_that_outgrow_their_reference_in_either_half(dev):
    """Ordinary steps (no mask) in which some row's scores rise far in the first or the second 64 keys of a step."""
    n, m = 150, 128 * 8
    q, k, v, _ = make(dev, [n], [m], 2, 2, False, seed=21, gain=0.5)
    up = torch.zeros((m,), device=dev)
    for at, height in ((128 * 2 + 3, 30.0), (128 * 3 + 70, 65.0), (128 * 5, 66.0), (128 * 6 + 64, 110.0)):
        up[at:] = height
    q[..., 0] = 0
    q[::3, :, 0] = 128 ** 0.5  # a row in three climbs, the others stay
    k[..., 0] = up[:, None].to(torch.bfloat16)
    for causal in (False, True):
        out, lse = mla.mla_prefill(q, k, v, cu_of([n], dev), cu_of([m], dev), causal=causal)
        check(out, lse, q, k, v, None, [n], [m], causal)
    assert mla.mla_device_status() == 0


def test_a_partition_of_another_call_is_reported(dev):
    """Made for the other mask, or for more heads (of as many words): nothing is written, with cuts and without."""
    for lq, lk in (([70, 33], [70, 50]), ([64], [9000])):
        q, k, v, kr = make(dev, lq, lk, 4, 2, True)
        cq, ck = cu_of(lq, dev), cu_of(lk, dev)
        for heads, causal in (((4, 2), False), ((8, 4), True), ((4, 1), True)):
            md = mla.mla_get_metadata_prefill(cq, ck, q.shape[0], k.shape[0], *heads, causal=causal)
            out, lse = torch.full((q.shape[0], 4, 128), 5.0, dtype=torch.bfloat16, device=dev), torch.full((q.shape[0], 4), 5.0, device=dev)
            try:
                mla.mla_prefill(q, k, v, cq, ck, k_rope=kr, out=out, lse=lse, metadata=md)
            except ValueError:  # another number of words
                assert heads == (4, 1)
                continue
            assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
            assert (out == 5).all() and (lse == 5).all()
        md = mla.mla_get_metadata_prefill(cq, ck, q.shape[0], k.shape[0], 4, 2)
        out, lse = mla.mla_prefill(q, k, v, cq, ck, k_rope=kr, metadata=md)
        check(out, lse, q, k, v, kr, lq, lk, True)
        assert mla.mla_device_status() == 0
