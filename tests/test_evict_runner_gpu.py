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


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("elsewhere", [False, True])
def test_new_keys_do_not_inherit_an_evicted_keys_weight(kv8, elsewhere):
    """Evict, append a token into a slot or a page that held an evicted key, weigh with the call's defaults: its
    weight is its own probability (a row's probabilities over a head add up to 1)."""
    lens, kept, pool = [70, 90, 33], [40, 32, 20], 40
    db, cache = make(lens, 4, pool, kv8)
    if not kv8:   # finite scores
        db.kv_data.copy_(torch.randn(db.kv_data.shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda"))
    w = torch.rand(pool, HKV, P, device="cuda") * 100
    free = sorted(set(range(pool)) - set(db.host.kv_indices.tolist()))
    w[free] = 0
    if elsewhere:
        w[free[:3 + 2 + 2]] = 7   # the pages to fill: what their slots hold counts as nothing
    short, freed = runner.evict(db, w, kept, sink=1, window=4, cache=cache, pages=free if elsewhere else None)
    old = w.clone()
    held = torch.zeros(pool, P, dtype=torch.bool)
    for r, n in enumerate(kept):
        i = torch.arange(n)
        held[listed(short.host, r)[i // P], i % P] = True
    if elsewhere:
        held[db.host.kv_indices.long()] = True   # as they were
    assert not w.cpu()[~held.unsqueeze(1).expand(pool, HKV, P)].any()
    # a token more: the second request's in a page that was freed (or one more free one)
    spare = free[int(short.host.kv_indptr[-1]):] if elsewhere else freed.tolist()
    ids = [listed(short.host, r).tolist() for r in range(3)]
    ids = [x if len(x) * P > n else x + [spare.pop()] for x, n in zip(ids, kept)]
    one = dataclasses.replace(short.host, kv_lens=[n + 1 for n in kept], kv_indptr=torch.tensor(starts([len(x) for x in ids]), dtype=torch.int32),
                              kv_indices=torch.tensor(sum(ids, []), dtype=torch.int32),
                              kv_last_page_len=torch.tensor([n + 1 - (len(x) - 1) * P for x, n in zip(ids, kept)], dtype=torch.int32))
    grown = dataclasses.replace(short, host=one, kv_indptr=one.kv_indptr.cuda(), kv_indices=one.kv_indices.cuda(),
                                kv_last_page_len=one.kv_last_page_len.cuda())
    new = [torch.randn(3, HKV, D, device="cuda").to(BF) for _ in range(2)]
    if kv8:
        runner.append_kv8(grown, cache, *new, rotate_q=False)
        _, lse = runner.decode_kv8(grown, cache)
    else:
        runner.append_kv_axes(grown, *new, None, rotate_q=False)
        _, lse = runner.decode(grown)
    runner.add_key_weights(grown, lse, w, cache=cache)
    for r, n in enumerate(kept):
        page, slot = ids[r][n // P], n % P
        # From 0 to HQ / HKV: the codes' logits differ by hundreds, and exp(-104) is below half the least fp32, 2^-150.
        assert float(w[page, :, slot].min()) >= 0 and float(w[page, :, slot].max()) <= HQ // HKV + 1e-3
        gained = (rows(w.unsqueeze(-1), one, r) - rows(old.unsqueeze(-1), one, r)).double().sum((-2, -1))
        # A row's probabilities add up to 1: HQ / HKV rows a head, sums of 100 a key rounded in fp32 (n 100 2^-24).
        assert bool(((gained - HQ // HKV).abs() < 1e-3).all())


def test_an_eviction_is_remembered_where_keys_moved():
    db, _ = make([70, 90], 5, 20)
    rope, rows_ = api.make_rope_axes(1e4, D, [D // 2]), torch.zeros(2, HKV, D, dtype=BF, device="cuda")
    whole, freed = runner.evict(db, runner.zero_key_weights(20, HKV, P), [70, 200])
    assert not whole.host.moved and not freed.numel() and whole.host.kv_lens == [70, 90]
    short, _ = runner.evict(whole, runner.zero_key_weights(20, HKV, P), [70, 89])
    again, _ = runner.evict(short, runner.zero_key_weights(20, HKV, P), 1000)
    for x in (short, again):
        with pytest.raises(ValueError, match="position"):
            runner.append_kv_axes(x, rows_, rows_, rope)
    q = runner.append_kv_axes(short, rows_, rows_, rope, positions=ints([[69, 90]]))
    assert q.shape == db.q.shape
    torch.cuda.synchronize()


@pytest.mark.parametrize("budget", [2 ** 31, [10 ** 12, 20]])
def test_budgets_past_32_bits_keep_every_key(budget):
    db, _ = make([70, 90], 6, 20)
    short, freed = runner.evict(db, torch.rand(20, HKV, P, device="cuda"), budget, window=3)
    assert short.host.kv_lens == ([70, 90] if isinstance(budget, int) else [70, 20])
    assert sorted(short.host.kv_indices.tolist() + freed.tolist()) == sorted(db.host.kv_indices.tolist())
    torch.cuda.synchronize()
