"""GPU tests of the runner's eviction as a serving loop calls it: pages that requests share, what later appends and
weights find."""
import dataclasses

import numpy as np
import pytest
import torch

from paged_kv_cache_bsr_gb300 import api, runner, workloads as W
from length_util import BF, ints, starts

pytestmark = pytest.mark.gpu

P, HKV, HQ, D = 16, 2, 8, 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


def make(lens, seed, pool, kv8=False, shared=0):
    """(batch on the GPU, its 8-bit cache or None): decode rows; the first `shared` pages of every request are request 0's."""
    b = W.make_paged_batch(qo_lens=[1] * len(lens), kv_lens=lens, num_qo_heads=HQ, num_kv_heads=HKV, head_dim=D, page_size=P, dtype=BF,
                           seed=seed, pool_pages=pool)
    ids = b.kv_indices.clone()
    for r in range(1, len(lens)):
        s = int(b.kv_indptr[r])
        ids[s:s + shared] = ids[:shared]
    b = dataclasses.replace(b, kv_indices=ids)
    db, cache = runner.DeviceBatch.from_host(b), None
    if kv8:
        cache = runner.Kv8Cache.zeros(pool, HKV, P, D)
        g = torch.Generator("cuda").manual_seed(seed)
        cache.codes.view(torch.uint8).copy_(torch.randint(0, 0x7F, cache.codes.shape, generator=g, device="cuda", dtype=torch.uint8))
        cache.scales.copy_(torch.randint(120, 128, cache.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    return db, cache


def raw(db, cache):
    """The pool's bytes: [tensors], a head row's bytes or its exponent byte last."""
    return [db.kv_data.view(torch.uint8)] if cache is None else [cache.codes.view(torch.uint8), cache.scales.unsqueeze(-1)]


def listed(host, r):
    return host.kv_indices[int(host.kv_indptr[r]):int(host.kv_indptr[r + 1])].long()


def rows(t, host, r):
    """[..., keys]: request r's slots of a pool tensor [pages, ..., P, x] one behind another."""
    x = t[listed(host, r).cuda()].movedim(0, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])[..., :host.kv_lens[r], :]


def kept_of(w, n, sink, window):
    """Ascending kept indices of one list of weights by the definition: the last, the first, the heaviest."""
    n = min(n, w.size)
    tail = min(window, n)
    front = min(sink, n - tail)
    mid = np.arange(front, w.size - tail)
    best = mid[np.lexsort((mid, -w[mid].astype(np.float64)))][:n - tail - front]
    return sorted([*range(front), *range(w.size - tail, w.size), *best.tolist()])


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("stream", [False, True])
def test_shared_pages_are_shortened_into_others(kv8, stream):
    """Two requests over one prefix: their kept keys lie in pages of their own, the pages they had are as they were."""
    lens, budget, pool = [70, 90, 33], [40, 17, 33], 40
    db, cache = make(lens, 3, pool, kv8, shared=2)
    w = torch.rand(pool, HKV, P, device="cuda")
    free = sorted(set(range(pool)) - set(db.host.kv_indices.tolist()))[::-1]
    before, w0 = [t.clone() for t in raw(db, cache)], w.clone()
    err, s = ints([0]), torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="listed twice"):
        runner.evict(db, w, budget, cache=cache)
    short, freed = runner.evict(db, w, budget, sink=2, window=5, cache=cache, error=err, stream=s, pages=free)
    torch.cuda.synchronize()
    assert int(err) == 0 and short.host.kv_lens == [40, 17, 33]
    assert short.host.kv_indices.tolist() == free[:3 + 2 + 3] == short.kv_indices.tolist()
    assert freed.tolist() == sorted(set(db.host.kv_indices.tolist()))
    for t, t0 in zip(raw(db, cache), before):
        assert torch.equal(t[freed.long().cuda()], t0[freed.long().cuda()])
    assert torch.equal(w[freed.long().cuda()], w0[freed.long().cuda()])
    for r in range(3):
        old_w, new_w = rows(w0.unsqueeze(-1), db.host, r)[..., 0], rows(w.unsqueeze(-1), short.host, r)[..., 0]
        for h in range(HKV):
            keep = kept_of(old_w[h].cpu().numpy(), budget[r], 2, 5)
            assert torch.equal(new_w[h], old_w[h, keep])
            for t, t0 in zip(raw(db, cache), before):
                assert torch.equal(rows(t, short.host, r)[:, h], rows(t0, db.host, r)[:, h][:, keep])
