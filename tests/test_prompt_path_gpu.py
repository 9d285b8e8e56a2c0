"""One attention layer from a prompt to a decoding step: pages assigned, heads and rows normalised and rotated, rows
placed, a first chunk and one behind its read-back context attended to, then a decoding step over the same cache.

Every stage is held to the formula on what it was given; at the end the two ways to attend (up-projected heads
over rows, absorbed heads over the cache) have to agree on the last token.
"""
import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
import oracle
from mla_decode_attention_latent_gb300 import workloads as W
from tests import parity
from tests.test_norm_rope_gpu import formula, near
from tests.test_prefill_gpu import check

pytestmark = pytest.mark.gpu
PAGE, LATENT, ROPE, HEAD = 64, 512, 64, 128


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


def bf(*shape, g, gain=1.0):
    return (gain * torch.randn(shape, generator=g)).to(torch.bfloat16).cuda()


def i32(v, dev):
    return torch.tensor(list(v), dtype=torch.int32, device=dev)


def cu_of(lens):
    return torch.nn.functional.pad(torch.tensor(lens).cumsum(0), (1, 0)).to(torch.int32).cuda()


class Layer:
    """Weights of one layer (h heads) and what a server keeps of its requests."""

    def __init__(self, h, b, nblk, width, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.h, self.hidden = h, 256
        self.w_q = bf(self.hidden, h * (HEAD + ROPE), g=g, gain=self.hidden ** -0.5)
        self.w_kv = bf(self.hidden, LATENT + ROPE, g=g, gain=self.hidden ** -0.5)
        self.w_up = bf(LATENT, h * 2 * HEAD, g=g, gain=LATENT ** -0.5)  # keys and values of a head side by side
        self.kv_norm, self.q_norm = bf(LATENT, g=g) * 0.1 + 1, bf(HEAD + ROPE, g=g) * 0.1 + 1
        self.turns = mla.mla_rope_turns(ROPE, 10000.0, 40.0, 4096)
        self.scale, self.mscale = (HEAD + ROPE) ** -0.5, 1.1
        dev = torch.device("cuda", 0)
        self.cache = torch.zeros((nblk, PAGE, 1, LATENT + ROPE), dtype=torch.bfloat16, device=dev)
        self.table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros((b,), dtype=torch.int32, device=dev)
        self.free, self.left = torch.randperm(nblk, generator=g).to(torch.int32).to(dev), i32([nblk], dev)

    def rows(self, x, counts, pad):
        """Pages, rotated queries [n, h, 192], and the new rows in the cache; returns (q, latent, k_rope, positions, slots)."""
        n = x.shape[0]
        self.before = self.lens.clone()
        _, pos, slots = mla.mla_assign_pages(self.lens, cu_of(counts), self.table, self.free, self.left, n, new_seqlens=self.lens)
        q = (x @ self.w_q).view(n, self.h, HEAD + ROPE)
        want, bound = formula(q, pos, self.turns, self.q_norm, 1e-6, True, self.mscale)
        mla.mla_norm_rope(q, pos, self.turns, weight=self.q_norm, interleaved=True, rope_scale=self.mscale, out=q)
        near(q, want, bound)
        kv = x @ self.w_kv
        kept = torch.empty_like(kv)
        mla.mla_norm_rope_cache_write(kv[:, :LATENT], kv[:, LATENT:], pos, self.turns, slots, self.cache, weight=self.kv_norm, interleaved=True,
                                      rope_scale=self.mscale, latent_out=kept[:, :LATENT], k_rope_out=kept[:, LATENT:])
        lat, lb = formula(kv[:, None, :LATENT], None, None, self.kv_norm, 1e-6, False, 1.0)
        rope, rb = formula(kv[:, None, LATENT:], pos, self.turns, None, 0, True, self.mscale)
        near(kept, torch.cat([lat, rope], -1)[:, 0], torch.cat([lb, rb], -1)[:, 0])
        live = slots >= 0
        assert int(live.sum()) == sum(counts)
        assert torch.equal(self.cache.view(-1, LATENT + ROPE)[slots[live]], kept[live])
        return q, kept[:, :LATENT], kept[:, LATENT:], pos, slots

    def up(self, latent):
        both = (latent @ self.w_up).view(-1, self.h, 2 * HEAD)
        return both[..., :HEAD], both[..., HEAD:]


def test_from_a_prompt_to_a_decoding_step(dev):
    mla.mla_device_status()
    h, b = 16, 3
    layer = Layer(h, b, 24, 12)
    g = torch.Generator().manual_seed(9)
    # a first chunk of every prompt, in a buffer with room behind it
    first, pad = [70, 200, 1], 9
    x = bf(sum(first) + pad, layer.hidden, g=g)
    q, latent, k_rope, pos, _ = layer.rows(x, first, pad)
    assert layer.lens.tolist() == first and pos.tolist()[:71] == list(range(70)) + [0]
    k, v = layer.up(latent)
    cu = cu_of(first)
    out, lse = mla.mla_prefill(q, k, v, cu, cu, k_rope=k_rope, softmax_scale=layer.scale)
    check(out, lse, q, k, v, k_rope, first, first, True, scale=layer.scale)
    # the next chunk attends to its context too: the cached rows are read back and up-projected
    second = [130, 1, 63]
    x = bf(sum(second), layer.hidden, g=g)
    q, _, _, pos, _ = layer.rows(x, second, 0)
    total = [a + c for a, c in zip(first, second)]
    assert layer.lens.tolist() == total and pos.tolist() == [p for a, c in zip(first, second) for p in range(a, a + c)]
    cu_q, cu_k = cu_of(second), cu_of(total)
    latent, k_rope = mla.mla_cache_read(layer.cache, layer.table, torch.zeros_like(layer.lens), sum(total), cu_rows=cu_k)
    k, v = layer.up(latent)
    out, lse = mla.mla_prefill(q, k, v, cu_q, cu_k, k_rope=k_rope, softmax_scale=layer.scale)
    check(out, lse, q, k, v, k_rope, second, total, True, scale=layer.scale)
    # the last token of each prompt again, as a decoding step sees it: absorbed heads over the cache
    last = (cu_q[1:] - 1).long()
    w = layer.w_up.view(LATENT, h, 2 * HEAD)
    absorbed = torch.cat([torch.einsum("bhd,lhd->bhl", q[last][..., :HEAD].float(), w[..., :HEAD].float()), q[last][..., HEAD:].float()], -1)
    absorbed = absorbed.to(torch.bfloat16)[:, None].contiguous()
    md, ns = mla.mla_get_metadata(layer.lens, h, 1)
    o, dec_lse = mla.mla_decode_kvcache(absorbed, layer.cache, layer.table, layer.lens, LATENT, md, ns, softmax_scale=layer.scale)
    table = torch.where(layer.table < 0, 0, layer.table)
    want, want_lse = oracle.mla_decode(W.bf16_bits(absorbed.cpu()), W.bf16_bits(layer.cache.cpu()), table.cpu().numpy(), layer.lens.cpu().numpy(), LATENT,
                                       layer.scale, False)
    parity.assert_parity(o.float().cpu(), dec_lse.cpu(), want, want_lse)
    # the prompt's call has k and v rounded to bf16, the step the absorbed q: scores apart by at most e, weights by e^2e; then
    # p, v and o are rounded there, p and the latent o here, 2^-8 each and by norms
    again = torch.einsum("bhl,lhd->bhd", o[:, 0].double(), w[..., HEAD:].double())
    size = torch.linalg.matrix_norm(w[..., HEAD:].double().permute(1, 0, 2), 2)
    for i in range(b):
        keys = slice(int(cu_k[i]), int(cu_k[i + 1]))
        qn, kn = q[last[i]].double(), torch.cat([k[keys].double(), k_rope[keys].double()[:, None].expand(-1, h, -1)], -1)
        both = torch.cat([latent[keys], k_rope[keys]], -1).double()
        e = layer.scale * 2.0 ** -8 * (qn.norm(dim=-1) * kn.norm(dim=-1).amax(0) + absorbed[i, 0].double().norm(dim=-1) * both.norm(dim=-1).amax()) + 2.0 ** -10
        bound = (torch.expm1(2 * e) + 3 * 2.0 ** -8) * v[keys].double().norm(dim=-1).amax(0) + 2 * 2.0 ** -8 * size * latent[keys].double().norm(dim=-1).amax()
        assert bool(((again[i] - out[last[i]].double()).norm(dim=-1) <= bound).all())
        assert bool(((dec_lse[i, 0] - lse[last[i]]).abs() <= e).all())
    # the requests leave: every page comes back
    mla.mla_release_pages(layer.lens, torch.ones_like(layer.lens), layer.table, 24, layer.free, layer.left)
    assert layer.left.tolist() == [24] and sorted(layer.free.tolist()) == list(range(24))
    assert mla.mla_device_status() == 0


def test_a_chunk_whose_pages_do_not_suffice_waits(dev):
    """A request that gets no pages writes nothing, and is served when another one leaves."""
    layer = Layer(4, 2, 3, 4, seed=2)
    g = torch.Generator().manual_seed(3)
    x = bf(260, layer.hidden, g=g)
    cu = cu_of([130, 130])  # three pages each, three in all
    _, pos, slots = mla.mla_assign_pages(layer.lens, cu, layer.table, layer.free, layer.left, 260, new_seqlens=layer.lens)
    assert layer.lens.tolist() == [130, 0] and layer.left.tolist() == [0] and (slots[130:] == -1).all()
    kv = x @ layer.w_kv
    mla.mla_norm_rope_cache_write(kv[:, :LATENT], kv[:, LATENT:], pos, layer.turns, slots, layer.cache, weight=layer.kv_norm)
    assert int((layer.cache.view(-1, LATENT + ROPE) != 0).any(1).sum()) == 130
    mla.mla_release_pages(layer.lens, i32([1, 0], dev), layer.table, 3, layer.free, layer.left)
    assert layer.left.tolist() == [3] and layer.table[0].tolist() == [-1] * 4
    _, pos, slots = mla.mla_assign_pages(layer.lens, cu_of([0, 130]), layer.table, layer.free, layer.left, 130, new_seqlens=layer.lens)
    assert layer.lens.tolist() == [0, 130] and (slots >= 0).all()
    assert mla.mla_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_steps_are_those_of_eager_calls(dev, fp8):
    """A decoding step (pages, queries, rows, attention) captured once and replayed, sequences crossing page bounds."""
    b, h, nblk, width, steps = 3, 16, 16, 4, 70
    g = torch.Generator().manual_seed(4)
    x_q, x_kv = bf(b, h, LATENT + ROPE, g=g), bf(b, LATENT + ROPE, g=g)
    weight = bf(LATENT, g=g) * 0.1 + 1
    turns = mla.mla_rope_turns(ROPE)
    place = mla.mla_norm_rope_cache_write_fp8 if fp8 else mla.mla_norm_rope_cache_write
    decode = mla.mla_decode_kvcache_fp8 if fp8 else mla.mla_decode_kvcache

    def start():
        cache = torch.zeros((nblk, 64 * 580), dtype=torch.uint8, device=dev) if fp8 else torch.zeros((nblk, PAGE, 1, 576), dtype=torch.bfloat16, device=dev)
        s = dict(cache=cache, table=torch.full((b, width), -1, dtype=torch.int32, device=dev), lens=torch.zeros((b,), dtype=torch.int32, device=dev),
                 free=torch.randperm(nblk, generator=torch.Generator().manual_seed(5)).to(torch.int32).to(dev), left=i32([nblk], dev))
        s["lens"].zero_()
        _, pos, slots = mla.mla_assign_pages(s["lens"], cu_of([1, 60, 64]), s["table"], s["free"], s["left"], 125, new_seqlens=s["lens"])
        rows = bf(125, LATENT + ROPE, g=torch.Generator().manual_seed(6))
        place(rows[:, :LATENT], rows[:, LATENT:], pos, turns, slots, cache, weight=weight)
        return s

    def step(s, cu):
        _, pos, slots = mla.mla_assign_pages(s["lens"], cu, s["table"], s["free"], s["left"], b, new_seqlens=s["lens"])
        q = mla.mla_norm_rope(x_q, pos, turns)
        place(x_kv[:, :LATENT], x_kv[:, LATENT:], pos, turns, slots, s["cache"], weight=weight)
        md, ns = mla.mla_get_metadata(s["lens"], h, 1, num_parts=4)
        return decode(q[:, None], s["cache"], s["table"].clamp(min=0), s["lens"], LATENT, md, ns)

    cu = cu_of([1] * b)
    eager, replayed = start(), start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(start(), cu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o, lse = step(replayed, cu)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(steps):
        graph.replay()
        want, want_lse = step(eager, cu)
        assert torch.equal(o, want) and torch.equal(lse, want_lse), i
    assert replayed["lens"].tolist() == [71, 130, 134] and replayed["left"].tolist() == [nblk - 8]
    for name in ("cache", "table", "lens", "free"):
        assert torch.equal(eager[name], replayed[name]), name
    assert mla.mla_device_status() == 0
