"""Page assignment with bounds that make no sense here and there: every other sequence is served whole, every row is written."""
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


def plain(lens, cu, table, free, left, n):
    """The call by its definition: a sequence whose bounds descend, leave the rows or begin before the end of an earlier one is passed over."""
    table, after, pos, slots = [row[:] for row in table], [], [0] * n, [-1] * n
    asked = taken = end = status = 0
    for b, old in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        sense = 0 <= lo <= hi <= n
        good = sense and lo >= end and old >= 0 and old + hi - lo <= len(table[b]) * PAGE
        if sense:
            end = max(end, hi)
        if not good:
            status = _lib.MLA_DEVERR_SEQLEN
            after.append(max(old, 0))
            continue
        need = pages(old + hi - lo) - pages(old)
        asked += need
        if need and asked > left:
            after.append(old)
            continue
        for i in range(need):
            table[b][pages(old) + i] = free[left - 1 - taken]
            taken += 1
        for r in range(lo, hi):
            pos[r] = old + r - lo
            slots[r] = table[b][pos[r] // PAGE] * PAGE + pos[r] % PAGE
        after.append(old + hi - lo)
    return table, after, left - taken, pos, slots, status


def run(dev, lens, cu, n, width, seed=0, short=False):
    rng = random.Random(seed)
    pool = list(range(len(lens) * width + 50))
    rng.shuffle(pool)
    table = [[pool.pop() if c < pages(t) else -1 for c in range(width)] for t in lens]
    left = len(pool) // 2 if short else len(pool)
    want = plain(lens, cu, table, pool, left, n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    bt, num = i32(table), i32([left])
    # outputs of an earlier step, which a row that is not written would keep
    pos, slots = torch.full((n,), 77, dtype=torch.int32, device=dev), torch.full((n,), 77, dtype=torch.int64, device=dev)
    new, _, _ = mla.mla_assign_pages(i32(lens), i32(cu), bt, i32(pool), num, n, positions=pos, slots=slots)
    assert new.tolist() == want[1]
    assert slots.tolist() == want[4]
    assert pos.tolist() == want[3]
    assert bt.tolist() == want[0]
    assert num.tolist() == [want[2]]
    assert mla.mla_device_status() == want[5]


@pytest.mark.parametrize("cu,n", [
    ([0, 100, 3, 8], 8),        # an end past the rows: the sequence behind it has its own
    ([0, 4, -5, 8, 9], 9),      # a bound below 0
    ([0, 5, 3, 8], 8),          # descending: the last would begin inside the first
    ([0, 5, 3, 8, 11], 12),     # and one behind it that does not
    ([7, 2, 5, 5, 6], 6),       # a first bound that belongs to nobody
    ([0, -1, 2, 4], 4), ([-2, 1, 3], 3), ([0, 2, 2 ** 31 - 1, -2 ** 31, 2, 3], 5), ([4, 3, 2, 1, 0], 4), ([0, 3, 6], 5)])
def test_few(dev, cu, n):
    run(dev, [60 + 3 * b for b in range(len(cu) - 1)], cu, n, 3)
    run(dev, [0] * (len(cu) - 1), cu, n, 3)


def garbage(seed, b, most, count):
    rng = random.Random(seed)
    lens, cu = [rng.randint(0, 200) for _ in range(b)], [0]
    for _ in range(b):
        cu.append(cu[-1] + rng.randint(0, most))
    n = cu[-1] + 9
    for at in [rng.randrange(b + 1) for _ in range(count)]:
        cu[at] = rng.choice([-1, -2 ** 31, 2 ** 31 - 1, n + 1, 0, n, rng.randint(0, n), cu[at] + 1, max(0, cu[at] - 1)])
    return lens, cu, n


@pytest.mark.parametrize("b,most", [(5, 9), (128, 30), (100, 90)])
@pytest.mark.parametrize("seed", range(6))
def test_one_chunk(dev, b, most, seed):
    lens, cu, n = garbage(seed, b, most, 1 + seed)
    run(dev, lens, cu, n, pages(200 + most) + 1, seed, seed % 2 == 1)


@pytest.mark.parametrize("b,most", [(1025, 3), (2100, 20), (3000, 40)])
@pytest.mark.parametrize("seed", range(8))
def test_many_chunks(dev, b, most, seed):
    """More sequences than a CTA takes at once, senseless bounds at a chunk's ends and inside."""
    lens, cu, n = garbage(seed + b, b, most, 1 + 2 * seed)
    if seed % 2:
        cu[1024 - seed // 2 % 2] = (-5, n + 3, 2 ** 31 - 1, 0)[seed // 2]
    run(dev, lens, cu, n, pages(200 + most) + 1, seed, seed % 3 == 1)
