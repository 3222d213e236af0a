"""GPU parity of the accumulated attention weights of cached keys with their definition in 64 bits."""
import math

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api
from length_util import BF, FP, Paged, ints

pytestmark = pytest.mark.gpu

PAGES = [1, 2, 3, 5, 7, 8, 11, 16, 48, 64, 128, 256]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


def params(x, cap=0.0, causal=False):
    return api.make_params(x.hkv * x.group, x.hkv, x.d, x.P, x.dtype, x.d ** -0.5, cap, causal)


def run(x, lse, before, cap=0.0, causal=False, decay=1.0, weighed=None, q=None, **kw):
    w, err = before.clone(), ints([0])
    api.add_key_weights(params(x, cap, causal), x.indptr, x.indices, x.last, x.q if q is None else q, lse, x.kv, w, qo_indptr=x.qo,
                        kv_scales=x.scales, decay=decay, weighed_len=None if weighed is None else ints(weighed), error=err, **kw)
    return w, int(err)


def check(x, cap=0.0, causal=False, decay=1.0, weighed=None, lse=None, seed=0):
    causal_rows = causal and x.qo is not None
    lse = x.lse(x.d ** -0.5, cap, causal_rows) if lse is None else lse
    g = torch.Generator("cuda").manual_seed(seed)
    before = torch.rand(x.pool, x.hkv, x.P, generator=g, device="cuda") * 3
    if weighed is not None or decay == 0:   # what is not read may be anything
        for b, n in enumerate(x.kv_lens):
            page, slot = x.places(b, torch.arange(0 if decay == 0 else min(weighed[b], n), n, device="cuda"))
            before[page, :, slot] = float("nan")
    got, err = run(x, lse, before, cap, causal, decay, weighed)
    assert err == 0
    ref, bound = x.new_weights(lse, before, x.d ** -0.5, cap, causal_rows, decay, weighed)
    held = x.held[:, None, :].expand_as(got)
    assert torch.equal(got[~held], before[~held])   # slots that hold no key
    off = (got.double() - ref).abs()
    assert bool((off[held] <= bound[held]).all()), float((off - bound)[held].max())
    return got, ref


@pytest.mark.parametrize("P", PAGES)
def test_decode_step_over_page_sizes(P):
    """One row per request, lengths around the tiles' and the pages' edges, and empty requests."""
    lens = [1, 15, 16, 17, 0, P, P + 1, 300, 0, 129, 2 * P, 31]
    check(Paged(lens, P, 2, group=4, seed=P))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("group,hkv", [(1, 3), (2, 1), (4, 8), (8, 2)])
@pytest.mark.parametrize("kv8,cap", [(False, 0.0), (False, 30.0), (True, 0.0), (True, 30.0)])
def test_decode_step(d, dtype, group, hkv, kv8, cap):
    x = Paged([70, 1, 333, 16], 16, hkv, d=d, dtype=dtype, kv8=kv8, group=group, seed=group, spread=1.0 if kv8 else 0.0)
    got, _ = check(x, cap, decay=0.5, weighed=[69, 0, 332, 100])
    for b, n in enumerate(x.kv_lens):   # first step: a head's probabilities sum to 1
        page, slot = x.places(b, torch.arange(n, device="cuda"))
    w, _ = run(x, x.lse(x.d ** -0.5, cap), torch.zeros_like(got), cap)
    total = [w[x.places(b, torch.arange(n, device="cuda"))[0], :, x.places(b, torch.arange(n, device="cuda"))[1]].sum(0) for b, n in enumerate(x.kv_lens)]
    for t in total:
        assert (t - group).abs().max() < 2e-4 * group


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("causal,kv8,cap", [(True, False, 0.0), (True, True, 30.0), (False, False, 30.0), (False, True, 0.0)])
def test_prompts(dtype, group, causal, kv8, cap):
    """Ragged rows: whole prompts, prompts behind cached keys, more rows than keys, requests without either."""
    qo = [130, 64, 1, 200, 0, 70, 0, 129]
    kv = [130, 500, 257, 90, 40, 0, 0, 128]
    check(Paged(kv, 16, 2, dtype=dtype, kv8=kv8, qo_lens=qo, group=group, seed=group), cap, causal, decay=0.9,
          weighed=[0, 436, 256, 0, 40, 0, 0, 128])


@pytest.mark.parametrize("P", PAGES)
def test_prompts_over_page_sizes(P):
    check(Paged([300, 1, P, 129, 2 * P + 1], P, 2, qo_lens=[300, 1, P, 100, 33], group=8, seed=P), causal=True, decay=0.0)


@pytest.mark.parametrize("hkv,qo,kv", [(1, [700], [700]), (1, [1500], [130]), (2, [333, 20], [100, 900]), (1, [257], [5])])
@pytest.mark.parametrize("causal", [True, False])
def test_few_key_tiles_before_many_rows(hkv, qo, kv, causal):
    """Key tiles shared by the CTAs of a cluster, and equal bits of equal calls."""
    x = Paged(kv, 16, hkv, qo_lens=qo, group=8, seed=5)
    a, _ = check(x, causal=causal)
    b, _ = check(x, causal=causal)
    assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [2, 3, 4, 5, 33])
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_per_request(rows, kv8, d):
    """Draft tokens: several columns of the streaming kernel, up to where the other takes over; head_dim 64 stays."""
    check(Paged([200, rows, 77], 16, 2, d=d, kv8=kv8, qo_lens=[rows] * 3, group=4, seed=rows), causal=True)


@pytest.mark.parametrize("qo", [None, [60, 80, 33]])
def test_rows_without_lse_add_nothing(qo):
    """lse -inf takes a row out, whatever its query and its products are."""
    x = Paged([90, 80, 40], 16, 2, qo_lens=qo, group=2, seed=6)
    lse = x.lse(x.d ** -0.5)
    out = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    out[1] = True
    out[:, 1] = True
    lse[out] = -math.inf
    q = x.q.masked_fill(out.unsqueeze(-1), float("nan"))
    clean = x.q.masked_fill(out.unsqueeze(-1), 0)
    before = torch.zeros(x.pool, x.hkv, x.P, device="cuda")
    got, err = run(x, lse, before, q=q)
    x.q = clean
    ref, bound = x.new_weights(lse, before, x.d ** -0.5)
    held = x.held[:, None, :].expand_as(got)
    assert err == 0 and bool(((got.double() - ref).abs()[held] <= bound[held]).all())


@pytest.mark.parametrize("qo,causal", [(None, False), ([100, 70], True)])
def test_nan_lse_reaches_the_keys_that_its_row_sees(qo, causal):
    x = Paged([100, 70], 16, 2, qo_lens=qo, group=4, seed=7)
    lse = x.lse(x.d ** -0.5, causal=causal)
    row = 0 if qo is None else 40
    lse[row, 5] = float("nan")    # a head of kv head 1
    got, _ = run(x, lse, torch.zeros(x.pool, x.hkv, x.P, device="cuda"), causal=causal)
    page, slot = x.places(0, torch.arange(100, device="cuda"))
    w = got[page, :, slot]
    seen = 41 if causal else 100
    assert torch.isnan(w[:seen, 1]).all() and torch.isfinite(w[seen:, 1]).all() and torch.isfinite(w[:, 0]).all()
    page, slot = x.places(1, torch.arange(70, device="cuda"))
    assert torch.isfinite(got[page, :, slot]).all()


@pytest.mark.parametrize("qo", [None, [40, 70, 50]])
def test_bad_arrays_are_flagged_and_skipped(qo):
    x = Paged([100, 70, 50], 16, 2, qo_lens=qo, group=8, seed=8)
    lse = x.lse(x.d ** -0.5)
    before = torch.rand(x.pool, x.hkv, x.P, device="cuda")
    good, err = run(x, lse, before)
    assert err == 0
    keep = x.indices.clone()
    for bad in (-1, x.pool, 2 ** 31 - 1):
        x.indices[2] = bad
        got, err = run(x, lse, before)
        same = torch.ones(x.pool, dtype=torch.bool, device="cuda")
        same[keep[2].long()] = False
        assert err == 1 and torch.equal(got[same], good[same]) and torch.equal(got[~same], before[~same])
        x.indices.copy_(keep)
    page, slot = x.places(2, torch.arange(50, device="cuda"))
    for name, at, value in (("last", 1, 0), ("last", 1, 17), ("indptr", 3, 10 ** 6), ("indptr", 2, -5)) + (() if qo is None else (("qo", 3, 10 ** 6), ("qo", 1, -1))):
        arr = getattr(x, name)
        was = int(arr[at])
        arr[at] = value
        got, err = run(x, lse, before)
        assert err & 16 and torch.isfinite(got[x.held[:, None, :].expand_as(got)]).all(), name
        arr[at] = was


def test_other_stream_and_capture_with_new_lengths():
    """A captured call follows the arrays: lengths, pages and rows written before a replay."""
    x = Paged([300, 290], 16, 2, group=4, seed=9)
    lse = x.lse(x.d ** -0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    before = torch.zeros(x.pool, x.hkv, x.P, device="cuda")
    a, _ = run(x, lse, before)
    with torch.cuda.stream(s):
        b, _ = run(x, lse, before)
    s.synchronize()
    assert torch.equal(a, b)
    w, err = before.clone(), ints([0])
    graph = torch.cuda.CUDAGraph()
    call = lambda: api.add_key_weights(params(x), x.indptr, x.indices, x.last, x.q, lse, x.kv, w, error=err)
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    w.zero_()
    graph.replay()
    assert torch.equal(w, a)
    x.kv_lens = [300, 281]
    x.last[1] = 281 - 17 * 16   # a page fewer
    x.indptr[2] = int(x.indptr[2]) - 1
    lse.copy_(x.lse(x.d ** -0.5))
    w.zero_()
    graph.replay()
    ref, bound = x.new_weights(lse, before, x.d ** -0.5)
    assert int(err) == 0 and bool(((w.double() - ref).abs() <= bound + 1e-30).all())


def test_pool_past_4_gib():
    """Offsets past 32 bits: the last pages of a pool of 5 GiB."""
    P, hkv, d = 16, 8, 128
    pool = 5 * 2 ** 30 // (2 * hkv * P * d * 2) + 1
    x = Paged([200, 45], P, hkv, group=4, seed=10)
    big = torch.zeros(pool, 2, hkv, P, d, dtype=BF, device="cuda")
    to = torch.arange(pool - x.indices.numel(), pool, device="cuda")
    big[to] = x.kv[x.indices.long()]
    small = torch.zeros(x.pool, hkv, P, device="cuda")
    lse = x.lse(d ** -0.5)
    a, _ = run(x, lse, small)
    w = torch.zeros(pool, hkv, P, device="cuda")
    api.add_key_weights(params(x), x.indptr, to.to(torch.int32), x.last, x.q, lse, big, w)
    assert torch.equal(w[to], a[x.indices.long()]) and not w[:pool - x.indices.numel()].any()


@pytest.mark.parametrize("batch", [1, 31, 40, 128, 129, 200])
@pytest.mark.parametrize("bad", [False, True])
def test_many_prompts_of_very_different_lengths(batch, bad):
    """Key tiles in the order of their places up to 128 requests, in request order beyond; a request with bad
    arrays is left out and flagged, the others are as they were."""
    lens = [(37 * i * i + 5) % 700 if i % 7 else 0 for i in range(1, batch + 1)]
    x = Paged(lens, 16, 2, qo_lens=lens, group=4, seed=batch)
    got, _ = check(x, causal=True)
    if bad:
        b = max(range(batch), key=lambda i: lens[i])
        lse = x.lse(x.d ** -0.5, 0.0, True)
        before = torch.zeros_like(got)
        good, err = run(x, lse, before, causal=True)
        assert err == 0
        x.last[b] = 17
        w, err = run(x, lse, before, causal=True)
        page, _ = x.places(b, torch.arange(lens[b], device="cuda"))
        good[page] = 0
        assert err == 16 and torch.equal(w, good)


@pytest.mark.parametrize("kv8", [False, True])
def test_no_rows_only_decay(kv8):
    """A call without a row, as a captured step with nothing new has: the weights decay, new keys start at 0."""
    x = Paged([40, 17], 16, 2, kv8=kv8, qo_lens=[0, 0], group=4, seed=3)
    before = torch.rand(x.pool, 2, 16, device="cuda")
    lse = torch.empty(0, 8, device="cuda")
    got, err = run(x, lse, before, causal=True, decay=0.5, weighed=[30, 17])
    want = torch.where(x.held[:, None, :], before * 0.5, before)
    page, slot = x.places(0, torch.arange(30, 40, device="cuda"))
    want[page, :, slot] = 0
    assert err == 0 and torch.equal(got, want)
