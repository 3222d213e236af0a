"""Refusals of the prefill over packed keys and values, and its plan, without a GPU."""
import ctypes

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api

INVALID, BAD_INDEX, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    return api.load()


def host_plan(lib, kind=api.PLAN_PREFILL_RAGGED, hq=8, hkv=2, d=128, page=1, batch=4, rows=1000, keys=1000, dtype=api.PKV_BF16):
    h = ctypes.c_void_p()
    p = api.Params(hq, hkv, d, page, dtype, 0.1, 0.0, 1)
    st = lib.pkv_plan_create_host(ctypes.byref(h), kind, ctypes.byref(p), ctypes.byref(api.Limits(batch, rows, keys)), 152)
    return st, h


def compute(lib, h, qo, kv, rows):
    ws = torch.zeros(api.plan_workspace_bytes(h)[1] + 64, dtype=torch.uint8)
    at = ws.data_ptr() + (-ws.data_ptr()) % 64
    ip = lambda x: None if x is None else (ctypes.c_int32 * len(x))(*x)
    return lib.pkv_plan_compute(h, len(kv) - 1, ip(qo), ip(kv), None, None, rows, at, ws.numel() - 64)


@pytest.mark.parametrize("kw,st", [(dict(), 0), (dict(page=16), INVALID), (dict(d=64), UNSUPPORTED), (dict(hq=6), UNSUPPORTED),
                                   (dict(hq=7), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(hq=16, hkv=1), UNSUPPORTED)])
def test_plans(lib, kw, st):
    got, h = host_plan(lib, **kw)
    assert got == st
    if h:
        api.plan_destroy(h)


def test_plan_steps(lib):
    _, h = host_plan(lib)
    assert compute(lib, h, [0, 3, 300], [0, 3, 300], 300) == 0
    work = api.plan_get_work(h)
    assert sorted(work[:, 1].unique().tolist()) == [0, 1] and int(work[:, 6].max()) == 297
    assert compute(lib, h, [0, 3, 300], [0, 0, 300], 300) == 0       # a request without keys
    assert compute(lib, h, [0, 3, 300], [0, 3, 300], 299) == BAD_INDEX   # fewer rows of k and v than keys
    assert compute(lib, h, [0, 3, 300], [0, 5, 3], 300) == BAD_INDEX
    assert compute(lib, h, [0, 3, 300], [1, 3, 300], 300) == BAD_INDEX
    assert compute(lib, h, None, [0, 3, 300], 300) == INVALID
    assert compute(lib, h, [0, 1001], [0, 10], 10) == WORKSPACE
    assert compute(lib, h, [0, 10], [0, 1001], 2000) == WORKSPACE
    assert compute(lib, h, [0] * 6, [0] * 6, 10) == WORKSPACE
    api.plan_destroy(h)


def test_run_refuses_what_it_cannot_run(lib):
    """A plan that was never copied, plans of other kinds, and no plan."""
    buf = torch.zeros(4096, dtype=torch.uint8)
    p = ctypes.c_void_p(buf.data_ptr() + (-buf.data_ptr()) % 256)
    run = lambda h: lib.pkv_batch_prefill_ragged(h, p, 1024, p, 256, p, 256, p, p, p, None)
    assert run(None) == INVALID
    _, h = host_plan(lib)
    assert run(h) == INVALID
    assert lib.pkv_batch_prefill_paged(h, p, p, p, p, p, p, p, p, p, None) == INVALID
    api.plan_destroy(h)
    _, h = host_plan(lib, kind=api.PLAN_PREFILL, page=16)
    assert run(h) == INVALID
    api.plan_destroy(h)


def test_rows_of_the_binding():
    with pytest.raises(ValueError, match="CUDA"):
        api._rows(torch.zeros(4, 2, 128))
