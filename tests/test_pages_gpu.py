"""Pages taken from and returned to the free list: tables, lengths, positions and slots against a plain walk."""
import random

import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_status_left():
    mla.mla_device_status()
    yield


def pages(t):
    return -(-t // PAGE)


def plain(lens, counts, table, free, left, n):
    """The call by its definition, one sequence after the other."""
    table = [row[:] for row in table]
    after, pos, slots, r, asked, taken = [], [0] * n, [-1] * n, 0, 0, 0
    for b, (old, c) in enumerate(zip(lens, counts)):
        need = pages(old + c) - pages(old)
        asked += need
        ok = need == 0 or asked <= left
        if ok:
            for i in range(need):
                table[b][pages(old) + i] = free[left - 1 - taken]
                taken += 1
            for i in range(c):
                pos[r + i] = old + i
                slots[r + i] = table[b][(old + i) // PAGE] * PAGE + (old + i) % PAGE
        after.append(old + c if ok else old)
        r += c
    return table, after, left - taken, pos, slots


def make(seed, b, lo, hi, past, width=None):
    rng = random.Random(seed)
    lens = [rng.randint(0, past) for _ in range(b)]
    counts = [rng.randint(lo, hi) for _ in range(b)]
    width = width or pages(past + hi) + 1
    pool = list(range(b * width + 7))
    rng.shuffle(pool)
    table = [[-1] * width for _ in range(b)]
    for row, t in zip(table, lens):
        for c in range(pages(t)):
            row[c] = pool.pop()
    return lens, counts, table, pool


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def cu_of(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


# one sequence, a decoding batch, prompts, more sequences than a chunk of 1024, empty sequences
@pytest.mark.parametrize("b,lo,hi,past", [(1, 1, 1, 0), (1, 5000, 5000, 63), (64, 1, 1, 4096), (3, 0, 700, 130), (128, 0, 200, 64), (129, 1, 1, 640),
                                          (1023, 0, 3, 200), (1024, 1, 1, 128), (1025, 0, 2, 128), (2500, 0, 70, 64)])
@pytest.mark.parametrize("share", [1.0, 0.6, 0.0])
def test_assign(dev, b, lo, hi, past, share):
    lens, counts, table, free = make(b + hi, b, lo, hi, past)
    need = sum(pages(t + c) - pages(t) for t, c in zip(lens, counts))
    left = int(need * share)
    n = sum(counts) + 5
    want = plain(lens, counts, table, free, left, n)
    bt, num = i32(table, dev), i32([left], dev)
    new, pos, slots = mla.mla_assign_pages(i32(lens, dev), i32(cu_of(counts), dev), bt, i32(free, dev), num, n)
    assert bt.tolist() == want[0]
    assert new.tolist() == want[1]
    assert num.tolist() == [want[2]]
    assert pos.tolist() == want[3]
    assert slots.tolist() == want[4]
    assert mla.mla_device_status() == 0


def test_lengths_and_count_in_place_or_planned(dev):
    lens, counts, table, free = make(5, 1500, 0, 90, 200)
    left = sum(pages(t + c) - pages(t) for t, c in zip(lens, counts)) - 3
    want = plain(lens, counts, table, free, left, sum(counts))
    # planned: the count and the lengths are read only
    sl, num, out = i32(lens, dev), i32([left], dev), i32([0], dev)
    new = torch.zeros_like(sl)
    mla.mla_assign_pages(sl, i32(cu_of(counts), dev), i32(table, dev), i32(free, dev), num, sum(counts), num_free_out=out, new_seqlens=new)
    assert num.tolist() == [left] and sl.tolist() == lens and out.tolist() == [want[2]] and new.tolist() == want[1]
    # taken
    got = mla.mla_assign_pages(sl, i32(cu_of(counts), dev), i32(table, dev), i32(free, dev), num, sum(counts), new_seqlens=sl)
    assert got[0] is sl and sl.tolist() == want[1] and num.tolist() == [want[2]] and got[2].tolist() == want[4]


def test_no_rows_and_no_sequence_rows(dev):
    bt, num = i32([[-1, -1]], dev), i32([1], dev)
    new, pos, slots = mla.mla_assign_pages(i32([0], dev), i32([0, 0], dev), bt, i32([3, 9], dev), num, 0)
    assert new.tolist() == [0] and pos.numel() == slots.numel() == 0 and num.tolist() == [1]
    # rows before the first sequence and behind the last belong to none
    new, pos, slots = mla.mla_assign_pages(i32([0], dev), i32([2, 3], dev), bt, i32([3, 9], dev), num, 5)
    assert slots.tolist() == [-1, -1, 3 * 64, -1, -1] and pos.tolist() == [0] * 5 and num.tolist() == [0] and bt.tolist() == [[3, -1]]


def test_what_makes_no_sense_is_reported(dev):
    free = i32([4, 5, 6], dev)
    # past the table: not served, and the sequence behind it gets the top of the stack
    bt, num = i32([[0], [-1]], dev), i32([3], dev)
    new, pos, slots = mla.mla_assign_pages(i32([60, 0], dev), i32([0, 10, 11], dev), bt, free, num, 11)
    assert new.tolist() == [60, 1] and bt.tolist() == [[0], [6]] and slots.tolist() == [-1] * 10 + [6 * 64] and num.tolist() == [2]
    assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
    # bounds that descend or pass the rows, a negative length
    for lens, cu in (([0, 0], [0, 4, 2]), ([0, 0], [0, 1, 9]), ([-5, 0], [0, 1, 2]), ([0, 0], [-3, 1, 2])):
        bt, num = i32([[-1], [-1]], dev), i32([3], dev)
        mla.mla_assign_pages(i32(lens, dev), i32(cu, dev), bt, free, num, 4)
        assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN
    # a row lands on an entry that is no page
    bt, num = i32([[-1]], dev), i32([3], dev)
    new, pos, slots = mla.mla_assign_pages(i32([7], dev), i32([0, 1], dev), bt, free, num, 1)
    assert slots.tolist() == [-1] and mla.mla_device_status() == _lib.MLA_DEVERR_BLOCK_ID
    # a count beyond the list
    bt, num = i32([[-1]], dev), i32([8], dev)
    mla.mla_assign_pages(i32([0], dev), i32([0, 1], dev), bt, free, num, 1)
    assert mla.mla_device_status() == _lib.MLA_DEVERR_SEQLEN and bt.tolist() == [[6]]


@pytest.mark.parametrize("b,past", [(1, 200), (64, 4096), (1025, 130), (2100, 64)])
def test_release(dev, b, past):
    lens, _, table, free = make(b, b, 0, 0, past)
    rng = random.Random(3 * b)
    done = [rng.choice([0, 0, 1, 7]) for _ in range(b)]
    room = len(free) + sum(pages(t) for t in lens)
    fp = torch.full((room,), -9, dtype=torch.int32, device=dev)
    fp[:len(free)] = i32(free, dev)
    sl, bt, num = i32(lens, dev), i32(table, dev), i32([len(free)], dev)
    mla.mla_release_pages(sl, i32(done, dev), bt, 10 ** 6, fp, num)
    want = free + [table[i][c] for i in range(b) if done[i] for c in range(pages(lens[i]))]
    assert num.tolist() == [len(want)] and fp[:len(want)].tolist() == want
    assert sl.tolist() == [0 if d else t for d, t in zip(done, lens)]
    assert bt.tolist() == [[-1] * len(row) if d else row for d, row in zip(done, table)]
    assert mla.mla_device_status() == 0


def test_release_reports_bad_entries_and_overflow(dev):
    fp, num = torch.zeros((2,), dtype=torch.int32, device=dev), i32([0], dev)
    mla.mla_release_pages(i32([300], dev), i32([1], dev), i32([[8, -1, 99, 3, 7]], dev), 10, fp, num)
    assert mla.mla_device_status() == _lib.MLA_DEVERR_BLOCK_ID | _lib.MLA_DEVERR_SEQLEN
    assert fp.tolist() == [8, 3] and num.tolist() == [2]


def test_requests_come_and_go(dev):
    """Steps of a serving loop under one captured graph: no page is ever held twice, and all come back."""
    b, width, nblk, rng = 9, 8, 40, random.Random(1)
    sl, bt = torch.zeros((b,), dtype=torch.int32, device=dev), torch.full((b, width), -1, dtype=torch.int32, device=dev)
    fp, num = torch.arange(nblk, dtype=torch.int32, device=dev), i32([nblk], dev)
    cu, done = torch.zeros((b + 1,), dtype=torch.int32, device=dev), torch.zeros((b,), dtype=torch.int32, device=dev)
    pos, slots = torch.zeros((800,), dtype=torch.int32, device=dev), torch.zeros((800,), dtype=torch.int64, device=dev)

    def step():
        mla.mla_release_pages(sl, done, bt, nblk, fp, num)
        mla.mla_assign_pages(sl, cu, bt, fp, num, 800, new_seqlens=sl, positions=pos, slots=slots)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(25):
        lens = sl.tolist()
        gone = [1 if t > 200 and rng.random() < 0.5 else 0 for t in lens]
        done.copy_(i32(gone, dev))
        kept = [0 if g else t for g, t in zip(gone, lens)]
        counts = [min(rng.choice([1, 1, 40, 150]), width * PAGE - t, 80) for t in kept]
        cu.copy_(i32(cu_of(counts), dev))
        graph.replay()
        torch.cuda.synchronize()
        lens, table, free = sl.tolist(), bt.tolist(), fp.tolist()[:num.item()]
        held = [table[i][c] for i in range(b) for c in range(pages(lens[i]))]
        assert sorted(held + free) == list(range(nblk))
        at = [s for s in slots.tolist()[:sum(counts)] if s >= 0]
        assert len(set(at)) == len(at)
    assert mla.mla_device_status() == 0
