"""Calls from several threads at once, each on a stream of its own."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from tests import reference64 as R
from tests import test_blocks_gpu as blocks
from tests import test_tree_gpu as trees

pytestmark = pytest.mark.gpu

LENS = [1500, 300, 576]


def alike(want, got):
    return all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("what", ["blocks", "trees", "cache"])
def test_calls_from_several_threads(what):
    """Every call gives the bits that it gives alone, and one that raises in its thread fails the test."""
    dev = torch.device("cuda", 0)
    mla.mla_device_status()

    def job(h, fp8):
        if what == "blocks":
            q, cache, table, keys, scales = (t.to(dev) for t in blocks.make(LENS, 2, h, 576, fp8, seed=h))
            return lambda: blocks.decode(dev, q, cache, table, LENS, keys, scales, 6)
        if what == "trees":
            q, cache, table, sees = trees.make(LENS, 9, h, 576, fp8, seed=h)
            q, cache, table = q.to(dev), cache.to(dev), table.to(dev)
            return lambda: trees.decode(dev, q, cache, table, LENS, sees)
        g = torch.Generator().manual_seed(h)
        table, used = R.random_table(g, LENS)
        start = R.random_cache(g, used, 576, fp8).to(dev)
        table, x = table.to(dev), torch.randn((3 * h, 576), generator=g).to(torch.bfloat16).to(dev)
        at = torch.tensor([0, 64, 130], dtype=torch.int32, device=dev)
        lens = torch.tensor(LENS, dtype=torch.int32, device=dev)
        write = mla.mla_cache_write_fp8 if fp8 else mla.mla_cache_write
        read = mla.mla_cache_read_fp8 if fp8 else mla.mla_cache_read
        update = mla.mla_update_page_keys_fp8 if fp8 else mla.mla_update_page_keys

        def step():
            cache = start.clone()
            keys, scales = torch.zeros((used, 576), dtype=torch.int8, device=dev), torch.zeros((used,), device=dev)
            write(x[:, :512], x[:, 512:], cache, table, at)
            update(cache, table, lens, keys, scales)
            return (cache, keys, scales, *read(cache, table, at, 3 * h))
        return step

    jobs = [job(h, fp8) for h, fp8 in ((128, False), (128, True), (32, False), (32, True))]
    want = [j() for j in jobs]
    torch.cuda.synchronize()

    def work(i):
        stream = torch.cuda.Stream(dev)
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            got = [jobs[i]() for _ in range(20)]
            stream.synchronize()
            return [alike(want[i], g) for g in got]

    with ThreadPoolExecutor(len(jobs)) as pool:
        results = [f.result() for f in [pool.submit(work, i) for i in range(len(jobs))]]  # raises what a thread raised
    assert results == [[True] * 20] * len(jobs)
    assert mla.mla_device_status() == 0
