"""NaN in what a batch reads: it reaches the outputs and lse of every row that sees it, and nothing else, however
the plan splits the work.  Everything that does not see it keeps the bits of the call without it."""
import dataclasses

import numpy as np
import pytest
import torch

from paged_kv_cache_bsr_gb300 import api, runner
from kv8_util import batch

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


def cache_of(b, seed=0):
    """An 8-bit cache of finite codes for the batch's pool."""
    gen = torch.Generator("cuda").manual_seed(seed)
    shape = (b.num_pages, 2, b.num_kv_heads, b.page_size)
    codes = torch.randint(0, 256, (*shape, b.head_dim), generator=gen, dtype=torch.uint8, device="cuda")
    codes[(codes & 0x7F) == 0x7F] = 0x30
    return runner.Kv8Cache(codes.view(torch.float8_e4m3fn),
                           torch.randint(115, 120, shape, generator=gen, dtype=torch.uint8, device="cuda"))


def at(b, r, token):
    """(page, slot) of a request's token."""
    return int(b.kv_indices[int(b.kv_indptr[r]) + token // b.page_size]), token % b.page_size


def run(kind, b, plan, q, cache, kv):
    db = runner.DeviceBatch.from_host(b, kv_data=kv)
    db.q = q
    o, lse = {"decode8": lambda: runner.decode_kv8(db, cache, plan), "prefill8": lambda: runner.prefill_kv8(db, cache, plan),
              "decode16": lambda: runner.decode(db, plan), "prefill16": lambda: runner.prefill(db, plan),
              "mixed16": lambda: runner.mixed(db, plan)}[kind]()
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu()


KINDS = {"decode8": api.PLAN_DECODE_KV8, "prefill8": api.PLAN_PREFILL_KV8, "decode16": api.PLAN_DECODE,
         "prefill16": api.PLAN_PREFILL, "mixed16": api.PLAN_MIXED}


def same_bits(x, y):
    i = torch.int16 if x.element_size() == 2 else torch.int32
    return x.view(i) == y.view(i)


def check(kind, b, expect, keys, query_scale=1.0, dims=(5,), **plan_kw):
    """A NaN in each listed key, value and query element: (request, token, kv head), in turn."""
    g = b.num_qo_heads // b.num_kv_heads
    plan = runner.make_plan(b, KINDS[kind], **plan_kw)
    eight = kind.endswith("8")
    cache = cache_of(b) if eight else None
    kv = torch.empty(0) if eight else torch.nan_to_num(b.kv_data.float(), 0.0).to(b.dtype).cuda()
    runner.plan_batch(plan, b, num_pages=b.num_pages)
    expect(plan)
    q = (b.q.float() * query_scale).to(b.dtype).cuda()
    o, lse = run(kind, b, plan, q, cache, kv)
    assert torch.isfinite(o.float()).all() and not torch.isnan(lse).any()
    qo = b.qo_indptr.tolist()
    for r, token, h in keys:
        page, slot = at(b, r, token)
        heads = slice(h * g, (h + 1) * g)
        first = max(0, token - (b.kv_lens[r] - b.qo_lens[r])) if b.causal else 0   # the request's first row that sees it
        rows = slice(qo[r] + first, qo[r + 1])
        for which in (0, 1) if not b.causal else (0,):
            for dim in dims:
                if eight:
                    c8 = runner.Kv8Cache(cache.codes.view(torch.uint8).clone(), cache.scales)
                    c8.codes[page, which, h, slot, dim] = 0xFF
                    got, got_lse = run(kind, b, plan, q, c8, kv)
                else:
                    k2 = kv.clone()
                    k2[page, which, h, slot, dim] = NAN
                    got, got_lse = run(kind, b, plan, q, cache, k2)
                hit, hit_lse = torch.zeros(o.shape, dtype=torch.bool), torch.zeros(lse.shape, dtype=torch.bool)
                if which == 0:
                    hit[rows, heads], hit_lse[rows, heads] = True, True
                else:
                    hit[rows, heads, dim] = True
                what = f"{'KV'[which]} of request {r}, token {token}, head {h}"
                assert torch.isnan(got[hit]).all() and torch.isnan(got_lse[hit_lse]).all(), what
                assert same_bits(got, o)[~hit].all() and same_bits(got_lse, lse)[~hit_lse].all(), what
        row, head = qo[r + 1] - 1, h * g
        q2 = q.clone()
        q2[row, head, 7] = NAN
        got, got_lse = run(kind, b, plan, q2, cache, kv)
        hit = torch.zeros(lse.shape, dtype=torch.bool)
        hit[row, head] = True
        assert torch.isnan(got[hit]).all() and torch.isnan(got_lse[hit]).all(), f"query {row}, head {head}"
        assert same_bits(got, o)[~hit].all() and same_bits(got_lse, lse)[~hit].all()


def split(plan):
    assert plan.info().num_merge > 0


def whole(plan):
    assert plan.info().num_merge == 0


def shared(plan):
    assert plan.info().num_merge == 0 and (plan.work()[:, 6] == -2).any()


# --------------------------------------------------------------------------- decode over the 8-bit cache
# Queries of 300 times the size put most pieces' weights at zero: a NaN value behind such a weight still counts.
@pytest.mark.parametrize("scale", [1.0, 300.0])
@pytest.mark.parametrize("g,d,dtype,cap", [(4, 128, BF, 0.0), (8, 64, FP, 0.0), (1, 128, BF, 9.0)])
def test_decode8_few_lists_in_many_pieces(g, d, dtype, cap, scale):
    """Several warps to a row of the merge, some with one piece or none."""
    b = batch([1, 1], [30000, 600], hq=2 * g, hkv=2, d=d, dtype=dtype, cap=cap, seed=g, extra=0)
    check("decode8", b, split, [(0, 17000, 0), (0, 29999, 1), (1, 0, 0), (1, 599, 1), (1, 300, 0)], scale)


@pytest.mark.parametrize("scale", [1.0, 300.0])
def test_decode8_many_lists_in_few_pieces(scale):
    """One warp to a row of the merge."""
    b = batch([1] * 71, [600] * 70 + [3000], hq=8, hkv=4, seed=3, extra=0)
    check("decode8", b, split, [(0, 0, 0), (69, 599, 3), (70, 1500, 2)], scale)


@pytest.mark.parametrize("scale", [1.0, 300.0])
@pytest.mark.parametrize("d,P", [(128, 16), (64, 5)])
def test_decode8_lists_shared_within_a_cta(d, P, scale):
    b = batch([1] * 5, [1, 33, 250, 128, 400], hq=8, hkv=2, d=d, P=P, seed=4, extra=0)
    check("decode8", b, shared, [(0, 0, 0), (2, 100, 1), (4, 399, 0), (4, 0, 1)], scale)


def test_decode8_whole_lists():
    b = batch([1] * 4, [1, 33, 250, 900], hq=8, hkv=2, seed=5, extra=0)
    check("decode8", b, whole, [(0, 0, 0), (2, 100, 1), (3, 899, 0)], split_kv=False)


def test_decode8_empty_requests_beside_a_nan():
    """A request without keys keeps o = 0 and lse = -inf."""
    b = batch([1] * 3, [0, 20000, 0], hq=8, hkv=2, seed=6, extra=0)
    check("decode8", b, split, [(1, 19999, 1), (1, 3, 0)])


# --------------------------------------------------------------------------- prefill
@pytest.mark.parametrize("kind", ["prefill8", "prefill16"])
@pytest.mark.parametrize("g,dtype,cap", [(4, BF, 0.0), (2, FP, 7.0)])
def test_prefill_whole_tiles(kind, g, dtype, cap):
    b = batch([30, 5], [100, 128], hq=2 * g, hkv=2, dtype=dtype, cap=cap, seed=g, extra=0)
    check(kind, b, whole, [(0, 0, 0), (0, 99, 1), (1, 64, 0)])


@pytest.mark.parametrize("kind", ["prefill8", "prefill16"])
def test_prefill_causal_whole_tiles(kind):
    """A NaN key reaches the rows from its own on (it is masked for those before)."""
    check(kind, batch([128] * 20, [128] * 20, hq=16, hkv=8, causal=True, seed=9, extra=0), whole, [(0, 60, 1), (19, 127, 7)])


@pytest.mark.parametrize("kind", ["prefill8", "prefill16"])
@pytest.mark.parametrize("g,dtype,cap", [(4, BF, 0.0), (1, FP, 7.0), (8, FP, 0.0)])
def test_prefill_split_over_the_keys(kind, g, dtype, cap):
    b = batch([40, 3], [3000, 700], hq=2 * g, hkv=2, dtype=dtype, cap=cap, seed=g, extra=0)
    check(kind, b, split, [(0, 0, 0), (0, 2999, 1), (1, 350, 0)])


@pytest.mark.parametrize("kind", ["prefill8", "prefill16"])
def test_prefill_causal_split_over_the_keys(kind):
    check(kind, batch([300, 70], [300, 200], hq=8, hkv=2, causal=True, seed=8, extra=0), split, [(0, 250, 1), (1, 150, 0)])


def test_prefill_small_pages_and_a_mixed_batch():
    check("prefill16", batch([40, 3], [900, 70], P=1, seed=10, extra=0), split, [(0, 5, 0), (1, 69, 1)])
    check("mixed16", batch([1, 1, 40], [30000, 600, 3000], seed=11, extra=0), split, [(2, 5, 0), (2, 2999, 1)])


@pytest.mark.parametrize("kind", ["prefill8", "prefill16"])
def test_prefill_nan_value_behind_a_weight_of_zero(kind):
    """Queries of 300 times the size: most pieces of a split row weigh nothing beside its largest logits."""
    b = batch([40, 3], [3000, 700], hq=8, hkv=2, seed=14, extra=0)
    check(kind, b, split, [(0, t, 0) for t in (0, 700, 1500, 2300, 2999)] + [(1, 350, 1)], 300.0)


# --------------------------------------------------------------------------- states merged by the caller
@pytest.mark.parametrize("dtype", [BF, FP, torch.float32])
def test_merged_states(dtype):
    """Every pair, and every triple, of a finite, an empty and a NaN state: NaN where one is NaN."""
    import itertools
    vals = {"finite": (1.5, 0.25), "low": (-2.0, -400.0), "empty": (0.0, -np.inf), "nan": (NAN, NAN)}
    for n in (2, 3):
        combos = list(itertools.product(vals, repeat=n))
        o = torch.tensor([[vals[c[k]][0] for c in combos] for k in range(n)])[:, :, None, None].expand(-1, -1, 2, 128)
        o = o.to(dtype).contiguous().cuda()                        # [states, rows, heads, dim]
        lse = torch.tensor([[vals[c[k]][1] for c in combos] for k in range(n)])[:, :, None].expand(-1, -1, 2).contiguous().cuda()
        outs = []
        o_n, l_n = torch.empty_like(o[0]), torch.empty_like(lse[0])
        api.merge_states(o.flatten(0, 1), lse.flatten(0, 1), n, o_n, l_n)
        outs.append((o_n, l_n))
        if n == 2:
            o_2, l_2 = torch.empty_like(o[0]), torch.empty_like(lse[0])
            api.merge_state(o[0], lse[0], o[1], lse[1], o_2, l_2)
            outs.append((o_2, l_2))
        torch.cuda.synchronize()
        for got, got_lse in outs:
            got, got_lse = got.float().cpu(), got_lse.cpu()
            for i, c in enumerate(combos):
                if "nan" in c:
                    assert torch.isnan(got[i]).all() and torch.isnan(got_lse[i]).all(), c
                elif set(c) == {"empty"}:
                    assert (got[i] == 0).all() and torch.isneginf(got_lse[i]).all(), c
                else:
                    top = "finite" if "finite" in c else "low"     # the other's weight is e^-400.25 = 0
                    assert (got[i] == vals[top][0]).all(), c
                    want = vals[top][1] + np.log(c.count(top))
                    assert (got_lse[i] - want).abs().max() <= 2 * np.finfo(np.float32).eps * abs(want), c


def test_cascade8_nan_query_beside_an_empty_suffix():
    """The prefix's NaN state merged with the empty state of a request without a suffix."""
    prefix = batch([4], [500], seed=12, extra=0)
    suffix = batch([1] * 4, [0, 40, 0, 7], seed=13, extra=prefix.num_pages)
    cache = cache_of(suffix)
    q = prefix.q.cuda()
    clean = None
    for nan in (False, True):
        if nan:
            q[0, 3, 1], q[1, 2, 0] = NAN, NAN
        dbs = [runner.DeviceBatch.from_host(x, kv_data=torch.empty(0)) for x in (prefix, suffix)]
        for db in dbs:
            db.q = q
        o, lse = (x.cpu() for x in runner.cascade_kv8(*dbs, cache))
        torch.cuda.synchronize()
        if not nan:
            clean = o, lse
            assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    hit = torch.zeros(lse.shape, dtype=torch.bool)
    hit[0, 3] = hit[1, 2] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert same_bits(o, clean[0])[~hit].all() and same_bits(lse, clean[1])[~hit].all()


# --------------------------------------------------------------------------- decode over the 16-bit cache
@pytest.mark.parametrize("g,P", [(4, 16), (1, 8), (8, 16), (2, 1), (8, 4)])
def test_decode16_split(g, P):
    """Groups of 8 on pages of 8 rows or more run on the prefill kernel."""
    b = batch([1, 1, 1], [20000, 600, 0], hq=2 * g, hkv=2, P=P, seed=g, extra=0)
    check("decode16", b, split, [(0, 17000, 0), (1, 0, 1), (1, 599, 0)])


def test_decode16_whole_lists_and_in_a_mixed_batch():
    b = batch([1] * 3, [1, 250, 900], hq=8, hkv=2, seed=5, extra=0)
    check("decode16", b, whole, [(0, 0, 0), (1, 100, 1), (2, 899, 0)], split_kv=False)
    check("mixed16", batch([1, 1, 40], [30000, 600, 3000], seed=11, extra=0), split, [(0, 20000, 0), (1, 599, 1)])
