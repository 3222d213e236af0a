"""Refusals of the key weights, the choice of kept keys and their move, without a GPU: the C calls refuse
before they ask for a device, the binding before it calls."""
import ctypes

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api, runner, workloads as W

OK, INVALID, UNSUPPORTED = 0, -1, -3
BIG = 2 ** 31


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    return api.load()


_BUF = torch.zeros(4096, dtype=torch.uint8)
AT = _BUF.data_ptr() + (-_BUF.data_ptr()) % 256


def weights_call(lib, hq=8, hkv=2, d=128, page=16, dtype=api.PKV_BF16, scale=0.1, batch=2, total_q=2, pages=9, kv_pages=4,
                 qo=None, indptr=AT, indices=AT, last=AT, weighed=None, q=AT, kv=AT, scales=None, lse=AT, w=AT, decay=1.0,
                 err=None, params=True):
    p = api.Params(hq, hkv, d, page, dtype, scale, 0.0, 1)
    return lib.pkv_add_key_weights(ctypes.byref(p) if params else None, batch, total_q, pages, kv_pages, qo, indptr, indices,
                                   last, weighed, q, kv, scales, lse, w, decay, err, None)


@pytest.mark.parametrize("kw,st", [
    (dict(params=False), INVALID), (dict(batch=-1), INVALID), (dict(total_q=-1), INVALID), (dict(pages=-1), INVALID),
    (dict(kv_pages=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(hq=7), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(decay=-0.1), INVALID), (dict(decay=1.1), INVALID), (dict(decay=float("nan")), INVALID),
    (dict(page=0), UNSUPPORTED), (dict(page=20), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(hq=6), UNSUPPORTED), (dict(hq=32), UNSUPPORTED), (dict(page=1 << 21), UNSUPPORTED),
    (dict(pages=BIG), INVALID), (dict(kv_pages=BIG), INVALID), (dict(total_q=BIG, qo=AT), INVALID),
    (dict(pages=2 ** 29), UNSUPPORTED),                                     # head rows past 32 bits
    (dict(total_q=3), INVALID),                                             # one row per request
    (dict(indptr=None), INVALID), (dict(indices=None), INVALID), (dict(last=None), INVALID), (dict(kv=None), INVALID),
    (dict(w=None), INVALID), (dict(q=None), INVALID), (dict(lse=None), INVALID),
    (dict(q=AT + 8), INVALID), (dict(kv=AT + 8), INVALID), (dict(lse=AT + 2), INVALID), (dict(w=AT + 2), INVALID),
    (dict(scales=AT + 2), INVALID), (dict(indptr=AT + 2), INVALID), (dict(indices=AT + 1), INVALID), (dict(last=AT + 2), INVALID),
    (dict(weighed=AT + 2), INVALID), (dict(qo=AT + 2), INVALID), (dict(err=AT + 2), INVALID),
    (dict(batch=0, total_q=0), OK), (dict(kv_pages=0, w=None), OK)])
def test_key_weights(lib, kw, st):
    assert weights_call(lib, **kw) == st


def select_call(lib, batch=2, hkv=2, page=16, pages=9, kv_pages=4, indptr=AT, indices=AT, last=AT, w=AT, budget=AT, sink=1,
                window=1, most=8, keep=AT, kept=AT, err=None):
    return lib.pkv_select_keys(batch, hkv, page, pages, kv_pages, indptr, indices, last, w, budget, sink, window, most, keep, kept, err, None)


TABLE = [(dict(batch=-1), INVALID), (dict(hkv=0), INVALID), (dict(pages=-1), INVALID), (dict(kv_pages=-1), INVALID),
         (dict(most=-1), INVALID), (dict(page=0), UNSUPPORTED), (dict(page=20), UNSUPPORTED), (dict(page=1 << 21), UNSUPPORTED),
         (dict(hkv=1 << 21), UNSUPPORTED), (dict(pages=BIG), INVALID), (dict(kv_pages=BIG), INVALID),
         (dict(batch=BIG - 1), UNSUPPORTED), (dict(indptr=None), INVALID), (dict(indices=None), INVALID), (dict(last=None), INVALID),
         (dict(keep=None), INVALID), (dict(kept=None), INVALID), (dict(indptr=AT + 2), INVALID), (dict(indices=AT + 2), INVALID),
         (dict(last=AT + 1), INVALID), (dict(w=AT + 2), INVALID), (dict(keep=AT + 2), INVALID), (dict(kept=AT + 2), INVALID),
         (dict(err=AT + 2), INVALID), (dict(batch=0), OK)]


@pytest.mark.parametrize("kw,st", TABLE + [(dict(sink=-1), INVALID), (dict(window=-1), INVALID), (dict(w=None), INVALID),
                                           (dict(budget=None), INVALID), (dict(budget=AT + 2), INVALID)])
def test_select(lib, kw, st):
    assert select_call(lib, **kw) == st


def compact_call(lib, batch=2, hkv=2, page=16, d=128, dtype=api.PKV_F16, pages=9, kv_pages=4, indptr=AT, indices=AT, last=AT, most=8,
                 keep=AT, kept=AT, to_pages=0, to_indptr=None, to=None, kv=AT, scales=None, w=AT, err=None, params=True):
    p = api.Params(hkv, hkv, d, page, dtype, 1.0, 0.0, 0)
    return lib.pkv_compact_paged_kv(ctypes.byref(p) if params else None, batch, pages, kv_pages, indptr, indices, last, most, keep,
                                    kept, to_pages, to_indptr, to, kv, scales, w, err, None)


@pytest.mark.parametrize("kw,st", TABLE + [
    (dict(params=False), INVALID), (dict(d=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(kv=None), INVALID), (dict(kv=AT + 8), INVALID),
    (dict(to=AT), INVALID), (dict(to_indptr=AT), INVALID), (dict(to_pages=-1), INVALID), (dict(to_pages=BIG), INVALID),
    (dict(to=AT + 2, to_indptr=AT), INVALID), (dict(to=AT, to_indptr=AT + 2), INVALID), (dict(pages=2 ** 29), UNSUPPORTED),
    (dict(most=0), OK), (dict(kv_pages=0), OK)])
def test_compact(lib, kw, st):
    assert compact_call(lib, **kw) == st


# ----------------------------------------------------------------------------- binding
def tensors(batch=2, hq=8, hkv=2, d=128, P=16, pages=6):
    i = lambda *x: torch.zeros(*x, dtype=torch.int32)
    return dict(kv_indptr=i(batch + 1), kv_indices=i(4), kv_last_page_len=i(batch), q=torch.zeros(batch, hq, d, dtype=torch.bfloat16),
                lse=torch.zeros(batch, hq), kv=torch.zeros(pages, 2, hkv, P, d, dtype=torch.bfloat16), weights=torch.zeros(pages, hkv, P),
                budget=i(batch), keep=i(batch, hkv, 5), kept_len=i(batch))


BF = torch.bfloat16
CASES = {
    "weights": [dict(kv_indptr=torch.zeros(4, dtype=torch.int32)), dict(kv_indptr=torch.zeros(3)), dict(kv_indices=torch.zeros(4, dtype=torch.int64)),
                dict(q=torch.zeros(3, 8, 128, dtype=BF)), dict(q=torch.zeros(2, 8, 64, dtype=BF)), dict(q=torch.zeros(2, 8, 128)),
                dict(lse=torch.zeros(2, 7)), dict(lse=torch.zeros(2, 8, dtype=BF)), dict(kv=torch.zeros(6, 2, 2, 8, 128, dtype=BF)),
                dict(kv=torch.zeros(6, 2, 2, 16, 128)), dict(weights=torch.zeros(5, 2, 16)), dict(weights=torch.zeros(6, 2, 16, dtype=BF)),
                dict(qo_indptr=torch.zeros(2, dtype=torch.int32)), dict(weighed_len=torch.zeros(3, dtype=torch.int32)),
                dict(weighed_len=torch.zeros(2)), dict(kv_scales=torch.zeros(6, 2, 2, 16, dtype=torch.uint8)), dict(error=torch.zeros(1)), dict()],
    "select": [dict(weights=torch.zeros(6, 2, 16, dtype=BF)), dict(weights=torch.zeros(6, 32)), dict(keep=torch.zeros(2, 3, 5, dtype=torch.int32)),
               dict(keep=torch.zeros(2, 2, 5, dtype=torch.int64)), dict(budget=torch.zeros(3, dtype=torch.int32)), dict(budget=torch.zeros(2)),
               dict(kept_len=torch.zeros(1, dtype=torch.int32)), dict(kv_last_page_len=torch.zeros(3, dtype=torch.int32)), dict()],
    "compact": [dict(kv=torch.zeros(6, 2, 16, 128, dtype=BF)), dict(kv=torch.zeros(6, 2, 2, 16, 128)), dict(kv=torch.zeros(6, 3, 2, 16, 128, dtype=BF)),
                dict(kv_scales=torch.zeros(6, 2, 2, 16, dtype=torch.uint8)), dict(weights=torch.zeros(6, 2, 8)),
                dict(keep=torch.zeros(3, 2, 5, dtype=torch.int32)), dict(kept_len=torch.zeros(3, dtype=torch.int32)),
                dict(dst_indptr=torch.zeros(3, dtype=torch.int32)), dict(dst_indices=torch.zeros(3, dtype=torch.int32)),
                dict(dst_indptr=torch.zeros(2, dtype=torch.int32), dst_indices=torch.zeros(3, dtype=torch.int32)), dict()]}


@pytest.mark.parametrize("call,at", [(c, i) for c, x in CASES.items() for i in range(len(x))])
def test_binding_refuses(lib, call, at):
    """Shapes, types, and (the last case of each) tensors that are not on the GPU."""
    t = {**tensors(), **CASES[call][at]}
    table = [t.pop(k) for k in ("kv_indptr", "kv_indices", "kv_last_page_len")]
    extra = {k: t[k] for k in ("qo_indptr", "weighed_len", "kv_scales", "error", "dst_indptr", "dst_indices") if k in t}
    with pytest.raises(ValueError):
        if call == "weights":
            api.add_key_weights(api.make_params(8, 2, 128, 16, BF, 0.1), *table, t["q"], t["lse"], t["kv"], t["weights"], **extra)
        elif call == "select":
            api.select_keys(*table, t["weights"], t["budget"], t["keep"], t["kept_len"], **extra)
        else:
            api.compact_paged_kv(*table, t["keep"], t["kept_len"], t["kv"], weights=t["weights"], **extra)


def test_evict_refuses_budgets():
    b = W.make_paged_batch(qo_lens=[1, 1], kv_lens=[5, 9], num_qo_heads=2, num_kv_heads=1, head_dim=64, page_size=16, dtype=BF, seed=1)
    db = type("HostOnly", (), {"host": b})()
    for budget in ([3], [3, -1], -2):
        with pytest.raises(ValueError, match="budget"):
            runner.evict(db, None, budget)
