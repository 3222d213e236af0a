"""Host arrays of a plan that are shorter than what is read of them are refused by the binding, without a GPU."""
import ctypes

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    return api.load()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("kind,page", [(api.PLAN_PREFILL_RAGGED, 1), (api.PLAN_PREFILL, 16), (api.PLAN_MIXED, 16), (api.PLAN_PREFILL_KV8, 16),
                                       (api.PLAN_DECODE, 16)])
def test_short_arrays_are_refused(lib, kind, page):
    h, p = ctypes.c_void_p(), api.Params(8, 2, 128, page, api.PKV_BF16, 0.1, 0.0, 1)
    assert lib.pkv_plan_create_host(ctypes.byref(h), kind, ctypes.byref(p), ctypes.byref(api.Limits(4, 100, 100)), 152) == 0
    room = torch.zeros(api.plan_workspace_bytes(h)[1] + 64, dtype=torch.uint8)
    ws = room[(-room.data_ptr()) % 64:]
    ragged, decode = kind == api.PLAN_PREFILL_RAGGED, kind == api.PLAN_DECODE
    good = dict(qo=None if decode else ints(0, 1, 5), kv=ints(0, 2, 6), ids=None if ragged else ints(0, 1, 2, 3, 4, 5),
                last=None if ragged else ints(3, 4))

    def compute(**kw):
        x = {**good, **kw}
        api.plan_compute(h, 2, x["qo"], x["kv"], x["ids"], x["last"], 10, ws)

    compute()
    bad = [("kv", ints(0, 2))] + ([] if decode else [("qo", ints(0, 5))]) + ([] if ragged else [("ids", ints(0, 1, 2, 3, 4)), ("last", ints(3))])
    for name, x in bad:
        with pytest.raises(ValueError, match="entr"):
            compute(**{name: x})
    compute(ids=None)
    api.plan_destroy(h)
