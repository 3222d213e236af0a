"""The 8-bit cache's calls beside what the plan, the pool and a graph may do around them."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_bsr_gb300 import api, runner
from kv8_util import EPS2, assert_attention, batch, quantised, to_cuda

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
P_EPS = {"decode": {BF: 2.0 ** -11, FP: 2.0 ** -11}, "prefill": EPS2}   # probabilities: fp16 / the operand type


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    oracle.build()
    api.load()
    torch.cuda.set_device(0)


def test_runs_read_the_tables_that_were_copied():
    """A plan computed on the host alone, between a plan and its run, leaves the run as it was."""
    big, small = batch([1] * 2, [20000, 300], seed=130, extra=0), batch([1], [40], seed=131, extra=0)
    rows_big, rows_small = batch([64], [4000], seed=132, extra=0), batch([2], [40], seed=133, extra=0)
    for kind, b, other in ((api.PLAN_DECODE_KV8, big, small), (api.PLAN_PREFILL_KV8, rows_big, rows_small)):
        prefill = kind == api.PLAN_PREFILL_KV8
        cache, _ = quantised(b, 1, poison=False)
        db, c = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0)), to_cuda(cache)
        plan = runner.make_plan(b, kind)
        outs = []
        for between in (False, True):
            runner.plan_batch(plan, b)
            assert plan.info().num_merge > 0
            if between:
                api.plan_compute(plan.handle, other.batch, other.qo_indptr if prefill else None, other.kv_indptr,
                                 other.kv_indices, other.kv_last_page_len, other.num_pages, plan.host_ws)
                assert plan.info().num_merge == 0
            o, lse = torch.full_like(db.q, 99.0), torch.full(db.q.shape[:2], 99.0, device="cuda")
            plan.run(db.q, c.codes, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o, lse, kv_scales=c.scales,
                     qo_indptr=db.qo_indptr if prefill else None)
            torch.cuda.synchronize()
            outs.append((o, lse))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_a_plan_that_was_never_copied_does_not_run():
    b = batch([1], [40], seed=134)
    cache, _ = quantised(b)
    db, c = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0)), to_cuda(cache)
    plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
    runner.plan_batch(runner.make_plan(b, api.PLAN_DECODE_KV8), b)
    api.plan_compute(plan.handle, 1, None, b.kv_indptr, b.kv_indices, b.kv_last_page_len, b.num_pages, plan.host_ws)
    with pytest.raises(api.PkvError) as e:
        api.batch_decode_paged_kv8(plan.handle, db.q, c.codes, c.scales, db.kv_indices, db.kv_indptr, db.kv_last_page_len,
                                   torch.zeros_like(db.q), None, plan.dev_ws)
    assert e.value.status == -1
