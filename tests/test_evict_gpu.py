"""GPU tests of the choice of kept keys and of their move, against their definitions, and of a run of
attention, weights, choice, move and decode together."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_bsr_gb300 import api, runner, workloads as W
from length_util import BF, FP, Paged, ints, starts

pytestmark = pytest.mark.gpu

PAGES = [1, 3, 8, 16, 48, 128]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    oracle.build()
    api.load()
    torch.cuda.set_device(0)


# ------------------------------------------------------------------------------ select
def chosen(w, n, sink, window):
    """The kept indices of one list of weights (float32 numpy), by the definition."""
    n = max(min(n, w.size), 0)
    tail = min(window, n)
    front = min(sink, n - tail)
    middle = np.arange(front, w.size - tail)
    x = w[middle].astype(np.float64) + 0.0
    order = sorted(middle.tolist(), key=lambda i: (math.isnan(w[i]), -(0.0 if math.isnan(w[i]) else float(w[i])), i))
    del x
    return sorted([*range(front), *range(w.size - tail, w.size), *order[:n - tail - front]])


def select(x, weights, budget, sink, window, max_keep=None):
    keep = torch.full((len(x.kv_lens), x.hkv, max(max_keep if max_keep is not None else max(budget), 0)), 77, dtype=torch.int32, device="cuda")
    kept, err = torch.full((len(x.kv_lens),), 77, dtype=torch.int32, device="cuda"), ints([0])
    api.select_keys(x.indptr, x.indices, x.last, weights, ints(budget), keep, kept, sink=sink, window=window, error=err)
    return keep.cpu().numpy(), kept.cpu().tolist(), int(err)


def check_select(x, weights, budget, sink=0, window=0, max_keep=None):
    keep, kept, err = select(x, weights, budget, sink, window, max_keep)
    assert err == 0
    for b, n in enumerate(x.kv_lens):
        page, slot = x.places(b, torch.arange(n, device="cuda"))
        w = weights[page, :, slot].cpu().numpy()
        want_n = max(min(budget[b], n, keep.shape[2]), 0)
        assert kept[b] == want_n
        for h in range(x.hkv):
            want = chosen(w[:, h], want_n, sink, window)
            assert keep[b, h, :want_n].tolist() == want, (b, h)
            assert (keep[b, h, want_n:] == -1).all()


@pytest.mark.parametrize("P", PAGES)
@pytest.mark.parametrize("sink,window", [(0, 0), (4, 16), (1, 1000)])
def test_select_over_page_sizes(P, sink, window):
    lens = [1, 5, 100, 0, 1025, 33, 700]
    x = Paged(lens, P, 3, d=64, seed=P)
    check_select(x, torch.rand(x.pool, 3, P, device="cuda"), [1, 3, 50, 10, 200, 33, 1000], sink, window)
    check_select(x, torch.rand(x.pool, 3, P, device="cuda"), [0, -5, 99, 2, 1024, 1, 7], sink, window)


@pytest.mark.parametrize("kind", ["equal", "few values", "signs", "nan", "inf", "denormal", "one digit"])
def test_select_of_difficult_weights(kind):
    """Ties go to the lower index; -0 is +0; NaN is the lowest; infinities are values."""
    x = Paged([400, 1500, 64], 16, 2, d=64, seed=1)
    g = torch.Generator("cuda").manual_seed(3)
    w = torch.randn(x.pool, 2, 16, generator=g, device="cuda")
    if kind == "equal":
        w.fill_(1.5)
    elif kind == "few values":
        w = (w * 2).round() / 2
    elif kind == "signs":
        w = torch.where(w > 0, 0.0, torch.where(w > -0.5, -0.0, w))
    elif kind == "nan":
        w[w > 0.2] = float("nan")
        w[w < -1] = -math.inf
    elif kind == "inf":
        w[w > 1] = math.inf
        w[w < -1] = -math.inf
    elif kind == "denormal":
        w = (w * 3).round() * 1e-45
    else:
        w = 1 + w.abs() * 1e-7
    for budget in ([200, 700, 10], [399, 1499, 63], [1, 1, 1]):
        check_select(x, w, budget, 2, 5)


def test_select_shared_by_a_cluster_and_past_shared_memory():
    """Long lists: eight CTAs a list, and lists far past the average that shared memory is sized for."""
    x = Paged([30001, 2], 16, 1, d=64, seed=2)
    w = (torch.randn(x.pool, 1, 16, device="cuda") * 8).round() / 8
    check_select(x, w, [3001, 1], 4, 64)
    x = Paged([40000] + [3] * 40, 16, 2, d=64, seed=3)
    check_select(x, torch.rand(x.pool, 2, 16, device="cuda"), [100] + [2] * 40, 1, 1)
    x = Paged([70000], 64, 8, d=64, seed=4)
    check_select(x, torch.rand(x.pool, 8, 64, device="cuda"), [5000], 4, 128)


def test_select_bounds_and_bad_arrays():
    x = Paged([100, 90, 80], 16, 2, d=64, seed=5)
    w = torch.rand(x.pool, 2, 16, device="cuda")
    check_select(x, w, [1000, 50, 3], 4, 8, max_keep=60)      # max_keep bounds the budget
    keep, kept, err = select(x, w, [5, 5, 5], 0, 0, max_keep=0)
    assert kept == [0, 0, 0] and err == 0
    good = select(x, w, [40, 40, 40], 1, 2)
    was = x.last.clone()
    x.last[1] = 17
    keep, kept, err = select(x, w, [40, 40, 40], 1, 2)
    assert err == 16 and kept == [40, 0, 40] and (keep[1] == -1).all()
    assert (keep[0] == good[0][0]).all() and (keep[2] == good[0][2]).all()
    x.last.copy_(was)
    x.indices[0] = x.pool
    keep, kept, err = select(x, w, [40, 40, 40], 1, 2)
    assert err == 1 and (keep[1:] == good[0][1:]).all()


# ----------------------------------------------------------------------------- compact
def keep_lists(x, counts, seed=0, always=0):
    g = torch.Generator("cuda").manual_seed(seed)
    most = max(counts, default=0)
    keep = torch.full((len(counts), x.hkv, most), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(counts):
        for h in range(x.hkv):
            i = torch.randperm(x.kv_lens[b], generator=g, device="cuda")[:n].sort()[0]
            if always:   # the first keys stay where they are
                i = torch.cat([torch.arange(min(always, n), device="cuda"), i[i >= always][:0]]) if n <= always else \
                    torch.cat([torch.arange(always, device="cuda"),
                               (always + torch.randperm(x.kv_lens[b] - always, generator=g, device="cuda")[:n - always]).sort()[0]])
            keep[b, h, :n] = i.to(torch.int32)
    return keep


def moved(x, keep, counts, t, dst=None):
    """t [pool, ..., hkv, P, ...] with the kept rows moved: t is kv (axis 2 = heads), scales or weights."""
    out = t.clone()
    for b, n in enumerate(counts):
        i = torch.arange(n, device="cuda")
        to, to_slot = x.places(b, i) if dst is None else (dst[1][int(dst[0][b]) + i // x.P].long(), i % x.P)
        for h in range(x.hkv):
            page, slot = x.places(b, keep[b, h, :n].long())
            if t.dim() == 3:
                out[to, h, to_slot] = t[page, h, slot]
            else:
                out[to, :, h, to_slot] = t[page, :, h, slot]
    return out


def check_compact(x, counts, in_place=True, weights=True, seed=0, always=0):
    keep = keep_lists(x, counts, seed, always)
    w = torch.rand(x.pool, x.hkv, x.P, device="cuda") if weights else None
    dst = None
    if not in_place:
        pages = [-(-n // x.P) for n in counts]
        free = torch.tensor(sorted(set(range(x.pool)) - set(x.indices.tolist())), dtype=torch.int32, device="cuda")
        assert free.numel() >= sum(pages)
        dst = (ints(starts(pages)), free[torch.randperm(free.numel(), device="cuda")][:sum(pages)].contiguous())
    raw = x.kv.view(torch.uint8) if x.scales is not None else x.kv.view(torch.int16)
    want = [moved(x, keep, counts, t, dst) for t in (raw, x.scales, w) if t is not None]
    err = ints([0])
    api.compact_paged_kv(x.indptr, x.indices, x.last, keep, ints(counts), x.kv, kv_scales=x.scales, weights=w,
                         dst_indptr=None if dst is None else dst[0], dst_indices=None if dst is None else dst[1], error=err)
    assert int(err) == 0
    for a, t in zip(want, [t for t in (raw, x.scales, w) if t is not None]):
        assert torch.equal(a, t)


@pytest.mark.parametrize("P", PAGES)
@pytest.mark.parametrize("d,kv8", [(64, False), (128, False), (64, True), (128, True)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(P, d, kv8, in_place):
    """Every row width, counts from none to all, and nothing but the kept slots written."""
    lens = [1, 40, 300, 0, 129, 2100, 77]
    x = Paged(lens, P, 3, d=d, kv8=kv8, seed=P, extra=3 if in_place else sum(-(-n // P) for n in lens) + 2)
    check_compact(x, [1, 13, 150, 0, 129, 1500, 1], in_place, weights=d == 128, seed=P)


@pytest.mark.parametrize("hkv,lens,counts", [(1, [9000], [6000]), (8, [5000], [4999]), (8, [700] * 40, [300] * 40), (2, [20000, 3], [50, 2])])
@pytest.mark.parametrize("kv8", [False, True])
def test_compact_in_place_over_many_rounds(hkv, lens, counts, kv8):
    """Column slices of 32 bytes up to whole rows, each over several rounds, most rows shifted by a few."""
    check_compact(Paged(lens, 16, hkv, kv8=kv8, seed=hkv), counts, seed=hkv)
    check_compact(Paged(lens, 16, hkv, kv8=kv8, seed=hkv), counts, seed=hkv, always=min(min(counts), 40))


def test_compact_nothing_to_move_and_bad_lists():
    x = Paged([100, 64], 16, 2, seed=6)
    w = torch.rand(x.pool, 2, 16, device="cuda")
    every = torch.arange(64, dtype=torch.int32, device="cuda").expand(2, 2, 64).contiguous()
    before = x.kv.clone()
    err = ints([0])
    api.compact_paged_kv(x.indptr, x.indices, x.last, every, ints([64, 64]), x.kv, weights=w, error=err)
    assert torch.equal(x.kv.view(torch.int16), before.view(torch.int16)) and int(err) == 0
    for kept in ([101, 3], [-1, 3], [65, 3]):        # past the keys, negative, past max_keep
        x.kv.copy_(before)
        err.zero_()
        keep = keep_lists(x, [3, 3], 1)
        keep = torch.nn.functional.pad(keep, (0, 61), value=-1)
        want = moved(x, keep, [0, 3], x.kv.view(torch.int16))
        api.compact_paged_kv(x.indptr, x.indices, x.last, keep, ints(kept), x.kv, error=err)
        assert int(err) == 16 and torch.equal(x.kv.view(torch.int16), want)
    x.kv.copy_(before)
    err.zero_()
    keep = keep_lists(x, [20, 20], 2)
    keep[0, 1, 19] = 100                             # no key of the request
    want = moved(x, keep.clamp(max=99), [20, 20], x.kv.view(torch.int16))
    page, slot = x.places(0, torch.tensor([19], device="cuda"))
    want[page, :, 1, slot] = before.view(torch.int16)[page, :, 1, slot]
    api.compact_paged_kv(x.indptr, x.indices, x.last, keep, ints([20, 20]), x.kv, error=err)
    assert int(err) == 16 and torch.equal(x.kv.view(torch.int16), want)
    # a destination with too few pages
    x.kv.copy_(before)
    err.zero_()
    api.compact_paged_kv(x.indptr, x.indices, x.last, keep_lists(x, [20, 20]), ints([20, 20]), x.kv, dst_indptr=ints([0, 1, 2]),
                         dst_indices=ints([x.pool - 1, x.pool - 2]), error=err)
    assert int(err) == 16 and torch.equal(x.kv.view(torch.int16), before.view(torch.int16))


def test_compact_captured_and_on_another_stream():
    x = Paged([500, 300], 16, 2, seed=7)
    keep, n = keep_lists(x, [200, 100], 3), ints([200, 100])
    before = x.kv.clone()
    want = moved(x, keep, [200, 100], x.kv.view(torch.int16))
    api.compact_paged_kv(x.indptr, x.indices, x.last, keep, n, x.kv)
    assert torch.equal(x.kv.view(torch.int16), want)
    s = torch.cuda.Stream()
    x.kv.copy_(before)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.compact_paged_kv(x.indptr, x.indices, x.last, keep, n, x.kv)
    s.synchronize()
    assert torch.equal(x.kv.view(torch.int16), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.compact_paged_kv(x.indptr, x.indices, x.last, keep, n, x.kv)
    for counts in ([200, 100], [7, 0]):
        n.copy_(ints(counts))
        x.kv.copy_(before)
        want = moved(x, keep, counts, x.kv.view(torch.int16))
        graph.replay()
        assert torch.equal(x.kv.view(torch.int16), want)


# --------------------------------------------------------------------------- together
def kept_reference(b, db, kv, keep, kept):
    """A batch whose heads hold only the kept keys: oracle attention per (request, head) list."""
    out = []
    for r in range(b.batch):
        pages = b.kv_indices[int(b.kv_indptr[r]):int(b.kv_indptr[r + 1])].long()
        x = kv[pages].permute(1, 2, 0, 3, 4).reshape(2, b.num_kv_heads, -1, b.head_dim)
        out.append(torch.stack([x[:, h, keep[r, h, :kept[r]].long()] for h in range(b.num_kv_heads)], 1))
    return out


@pytest.mark.parametrize("kv8", [False, True])
def test_prompt_to_bounded_decode(kv8):
    """Packed prompt attention, append, weights from the prompt's last rows and from decode steps, eviction
    after each, and decode over what is left: against attention over the kept keys in 64 bits."""
    qo = [300, 45, 130]
    b = W.make_paged_batch(qo_lens=qo, kv_lens=qo, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, dtype=BF, seed=5,
                           causal=True, pool_pages=60)
    db = runner.DeviceBatch.from_host(b)
    k_new, v_new = (t.cuda() for t in W.new_kv_rows(b, seed=6))
    o, lse = runner.prefill_ragged(db.q, k_new, v_new, b.qo_indptr, sm_scale=b.sm_scale)   # before anything is in pages
    cache = runner.Kv8Cache.zeros(b.num_pages, 2, 16, 128) if kv8 else None
    if kv8:
        runner.append_kv8(db, cache, k_new, v_new, rotate_q=False)
        _, lse = runner.prefill_kv8(db, cache)
    else:
        runner.append_kv(db, k_new, v_new, rotate_q=False)
        o2, lse2 = runner.prefill(db)
        # The two plans cut tiles differently.  Each output is off by at most half a step of itself and, of the
        # largest value, half a step of its probabilities and 4e-4 (their logits); so they differ by twice that.
        off = 2 * (2.0 ** -8 * (o2.double().abs() * 1.01) + (2.0 ** -8 + 4e-4) * v_new.double().abs().max())
        assert bool(((o.double() - o2.double()).abs() <= off).all()) and bool(((lse - lse2).abs() <= 8e-4).all())
    err = ints([0])
    weights = torch.full((b.num_pages, 2, 16), float("nan"), device="cuda")
    # the last 20 rows of each prompt weigh its keys
    last = [min(20, n) for n in qo]
    pick = torch.cat([torch.arange(e - n, e) for e, n in zip(b.qo_indptr[1:].tolist(), last)]).cuda()
    lb = dataclasses.replace(b, q=b.q[pick.cpu()], qo_indptr=torch.tensor(starts(last), dtype=torch.int32), qo_lens=last)
    ldb = dataclasses.replace(db, host=lb, q=db.q[pick], qo_indptr=lb.qo_indptr.cuda())
    runner.add_key_weights(ldb, lse[pick].contiguous(), weights, cache=cache, decay=0.0, error=err)
    values = lambda: db.kv_data.double() if not kv8 else torch.from_numpy(
        oracle.kv8_values(cache.codes.view(torch.uint8).cpu().numpy(), cache.scales.cpu().numpy())).cuda()
    step, steps = db, 3
    for i in range(steps):
        held = step.host
        before, kv_before = weights.clone(), values()
        lists = [[chosen(before[held.kv_indices[int(held.kv_indptr[r]):int(held.kv_indptr[r + 1])].long()].permute(1, 0, 2).reshape(2, -1)[h, :n]
                         .cpu().numpy(), min(100, n), 2, 8) for h in range(2)] for r, n in enumerate(held.kv_lens)]
        step, freed = runner.evict(step, weights, 100, sink=2, window=8, cache=cache, error=err)
        kept = step.host.kv_lens
        assert kept == [min(100, n) for n in held.kv_lens] and step.host.kv_indices.numel() == sum(-(-n // 16) for n in kept)
        assert sorted(freed.tolist() + step.host.kv_indices.tolist()) == sorted(held.kv_indices.tolist())
        keep = torch.full((b.batch, 2, max(kept)), -1)
        for r in range(b.batch):
            for h in range(2):
                keep[r, h, :kept[r]] = torch.tensor(lists[r][h])
        want = kept_reference(held, step, kv_before, keep.cuda(), kept)
        # decode one row per request over what is left
        g = torch.Generator("cuda").manual_seed(i)
        q = torch.randn(b.batch, 8, 128, generator=g, device="cuda").to(BF)
        one = dataclasses.replace(step.host, q=q.cpu(), qo_indptr=torch.arange(b.batch + 1, dtype=torch.int32), qo_lens=[1] * b.batch, causal=False)
        odb = dataclasses.replace(step, host=one, q=q, qo_indptr=one.qo_indptr.cuda())
        o, lse = runner.decode(odb) if not kv8 else runner.decode_kv8(odb, cache)
        for r in range(b.batch):
            kk, vv = (want[r][j].repeat_interleave(4, 0) for j in range(2))
            y = b.sm_scale * torch.einsum("hd,hkd->hk", q[r].double(), kk)
            ro = torch.einsum("hk,hkd->hd", torch.softmax(y, -1), vv)
            bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 4e-4) * vv.abs().max() + 2.0 ** -24
            assert bool(((o[r].double() - ro).abs() <= bound).all())
            assert (lse[r].double() - torch.logsumexp(y, -1)).abs().max() <= 4e-4
        runner.add_key_weights(odb, lse, weights, cache=cache, decay=0.9, error=err)
        # a token more for each request, in the last page's next slot or a freed page
        lens = [n + 1 for n in step.host.kv_lens]
        pages, free = [], freed.tolist()
        for r, n in enumerate(lens):
            ids = step.host.kv_indices[int(step.host.kv_indptr[r]):int(step.host.kv_indptr[r + 1])].tolist()
            pages.append(ids if len(ids) * 16 >= n else ids + [free.pop() if free else int(max(b.kv_indices)) + 1 + r])
        assert all(p < b.num_pages for ids in pages for p in ids)
        grown = dataclasses.replace(one, kv_lens=lens, kv_indptr=torch.tensor(starts([len(p) for p in pages]), dtype=torch.int32),
                                    kv_indices=torch.tensor(sum(pages, []), dtype=torch.int32),
                                    kv_last_page_len=torch.tensor([n - (len(p) - 1) * 16 for n, p in zip(lens, pages)], dtype=torch.int32))
        gdb = dataclasses.replace(odb, host=grown, kv_indptr=grown.kv_indptr.cuda(), kv_indices=grown.kv_indices.cuda(),
                                  kv_last_page_len=grown.kv_last_page_len.cuda())
        rows = lambda: torch.randn(b.batch, 2, 128, generator=g, device="cuda").to(BF)
        if kv8:
            runner.append_kv8(gdb, cache, rows(), rows(), rotate_q=False, error=err)
        else:
            runner.append_kv_axes(gdb, rows(), rows(), None, rotate_q=False, error=err)
        _, lse = runner.decode(gdb) if not kv8 else runner.decode_kv8(gdb, cache)
        runner.add_key_weights(gdb, lse, weights, cache=cache, weighed_len=ints([n - 1 for n in lens]), error=err)
        page = grown.kv_indices[[int(grown.kv_indptr[r]) + (n - 1) // 16 for r, n in enumerate(lens)]].long().cuda()
        assert torch.isfinite(weights[page, :, torch.tensor([(n - 1) % 16 for n in lens], device="cuda")]).all()
        step = gdb
    assert int(err) == 0


def test_a_shared_prefix_is_weighed_with_the_merged_lse():
    """Cascade: the prefix as one request of all rows, the suffixes apart, both with the merged lse, give what
    one call over whole lists (in pages of their own) gives."""
    cb = W.cascade_decode(seed=9, batch=6, prefix_len=256, suffix_lo=5, suffix_hi=40, num_qo_heads=8, num_kv_heads=2)
    kv = cb.full.kv_data.cuda()
    pre, suf = (runner.DeviceBatch.from_host(x, kv_data=kv) for x in (cb.prefix, cb.suffix))
    _, lse = runner.cascade(pre, suf)
    w = runner.zero_key_weights(cb.full.num_pages, 2, cb.full.page_size)
    err = ints([0])
    runner.add_key_weights(pre, lse, w, error=err)
    runner.add_key_weights(suf, lse, w, error=err)
    total = torch.zeros(cb.full.num_pages, 2, cb.full.page_size, device="cuda")
    for r in range(6):
        one = runner.DeviceBatch.from_host(W.sub_batch(cb.full, [r]), kv_data=kv)
        runner.add_key_weights(one, lse[r:r + 1].contiguous(), total, error=err)
    assert int(err) == 0
    assert (w - total).abs().max() <= 1e-5 * float(total.max())
    assert abs(float(w.double().sum()) - 6 * 8) < 1e-2


def small_batch(seed):
    qo = [120, 77]
    b = W.make_paged_batch(qo_lens=qo, kv_lens=qo, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, dtype=BF, seed=seed,
                           causal=True, pool_pages=20)
    db = runner.DeviceBatch.from_host(b)
    db.kv_data = torch.randn(db.kv_data.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(BF)
    return db


def shorten(db, stream=None):
    o, lse = runner.prefill(db, stream=stream)
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
        w = runner.zero_key_weights(db.host.num_pages, 2, 16)
    runner.add_key_weights(db, lse, w, stream=stream)
    short, freed = runner.evict(db, w, [50, 33], sink=1, window=4, stream=stream)
    return short, freed, w


def test_two_caches_on_two_streams_at_once():
    """Every step of two batches on streams of their own, beside each other, gives what one after the other gives."""
    want = []
    for seed in (1, 2):
        db = small_batch(seed)
        short, freed, w = shorten(db)
        want.append((db.kv_data, w, freed, short.kv_indices))
    batches, streams = [small_batch(s) for s in (1, 2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for db, s in zip(batches, streams):
        got.append(shorten(db, s))
    torch.cuda.synchronize()
    for db, (short, freed, w), (kv, w0, freed0, ids) in zip(batches, got, want):
        assert torch.equal(db.kv_data.view(torch.int16), kv.view(torch.int16)) and torch.equal(w, w0)
        assert torch.equal(freed, freed0) and torch.equal(short.kv_indices, ids) and short.host.kv_lens == [50, 33]


def test_a_choice_and_a_move_in_one_graph_follow_the_budgets():
    """select_keys and compact_paged_kv captured together, replayed with other budgets and weights."""
    x = Paged([300, 200], 16, 2, seed=11)
    w = torch.rand(x.pool, 2, 16, device="cuda")
    budget, kept = ints([100, 50]), ints([0, 0])
    keep = torch.empty(2, 2, 150, dtype=torch.int32, device="cuda")
    kv0 = x.kv.clone()

    def call():
        api.select_keys(x.indptr, x.indices, x.last, w, budget, keep, kept, sink=1, window=3)
        api.compact_paged_kv(x.indptr, x.indices, x.last, keep, kept, x.kv, weights=w)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n, seed in (([100, 50], 1), ([150, 1], 2), ([0, 149], 3)):
        budget.copy_(ints(n))
        w.copy_(torch.rand(w.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        x.kv.copy_(kv0)
        before = w.clone()
        graph.replay()
        for b in range(2):
            page, slot = x.places(b, torch.arange(x.kv_lens[b], device="cuda"))
            for h in range(2):
                want = chosen(before[page, h, slot].cpu().numpy(), n[b], 1, 3)
                assert keep[b, h, :n[b]].tolist() == want and int(kept[b]) == n[b]
        assert torch.equal(x.kv.view(torch.int16), moved(x, keep, n, kv0.view(torch.int16)))
        assert torch.equal(w, moved(x, keep, n, before))
