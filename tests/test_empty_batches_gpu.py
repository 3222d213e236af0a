"""Batches in which no request holds a key (their page tables are empty tensors, without an address), and batches
without a query row."""
import dataclasses

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api, runner
from kv8_util import batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


def cache_of(b):
    return runner.Kv8Cache.zeros(b.num_pages, b.num_kv_heads, b.page_size, b.head_dim)


RUNS = {"decode": lambda db, c: runner.decode(db), "decode_kv8": lambda db, c: runner.decode_kv8(db, c),
        "prefill": lambda db, c: runner.prefill(db), "prefill_kv8": lambda db, c: runner.prefill_kv8(db, c),
        "mixed": lambda db, c: runner.mixed(db)}


@pytest.mark.parametrize("name", sorted(RUNS))
@pytest.mark.parametrize("P,g", [(16, 4), (1, 4), (16, 8)])
def test_no_request_has_keys(name, P, g):
    b = batch([1, 1, 1] if name.startswith("decode") else [1, 40, 1], [0, 0, 0], hq=2 * g, hkv=2, P=P, extra=3)
    db = runner.DeviceBatch.from_host(b)
    assert db.kv_indices.numel() == 0
    o, lse = RUNS[name](db, cache_of(b))
    torch.cuda.synchronize()
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())


def test_a_cascade_whose_suffixes_are_all_empty():
    prefix = batch([4], [100], seed=1, extra=0)
    suffix = dataclasses.replace(batch([1] * 4, [0] * 4, seed=2, extra=prefix.num_pages), q=prefix.q)
    cache = cache_of(prefix)
    cache.codes.view(torch.uint8).random_(0, 0x70)
    cache.scales.fill_(116)
    dp, ds = (runner.DeviceBatch.from_host(x, kv_data=torch.empty(0)) for x in (prefix, suffix))
    o, lse = runner.cascade_kv8(dp, ds, cache)
    want, want_lse = runner.prefill_kv8(dp, cache)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("name", sorted(RUNS))
def test_no_query_rows(name):
    """No request at all (decode), or requests without new rows."""
    rows, keys = ([], []) if name.startswith("decode") else ([0, 0], [20, 3])
    b = batch(rows, keys, extra=2)
    o, lse = RUNS[name](runner.DeviceBatch.from_host(b), cache_of(b))
    torch.cuda.synchronize()
    assert o.shape[0] == 0 and lse.shape[0] == 0


def test_captured_calls_need_their_buffers():
    """A graph may be replayed with other batches: one captured without a page table, or without rows, is refused."""
    for lens in ([0, 0], []):
        b = batch([1] * len(lens), lens, extra=2)
        db, cache = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0)), cache_of(b)
        plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
        runner.plan_batch(plan, b)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        refused = None
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            mark = torch.zeros(1, device="cuda")
            try:
                runner.decode_kv8(db, cache, plan, stream=s)
            except api.PkvError as e:
                refused = e.status
            mark += 1
        assert refused == -1
