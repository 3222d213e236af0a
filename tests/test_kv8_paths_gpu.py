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


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_single_key_gives_its_value(kind, dtype):
    """Every code at scales over the type's range, past it and below its subnormals' step: what a row that sees
    one key gets is that key's value rounded to the type, and exact where the type holds it."""
    scales = np.arange(20, 240, 6) if dtype is BF else np.concatenate([np.arange(92, 148, 2), [85, 150, 200]])
    b = batch([1] * len(scales), [1] * len(scales), dtype=dtype, hq=8, hkv=2, seed=3, extra=0)
    codes, s8 = np.zeros((b.num_pages, 2, 2, 16, 128), np.uint8), np.full((b.num_pages, 2, 2, 16), 100, np.uint8)
    page = b.kv_indices[b.kv_indptr[:-1].long()].numpy()
    every = np.array([c for c in range(256) if c & 0x7F != 0x7F] + [0x30, 0xB0], np.uint8).reshape(2, 128)
    codes[page, 0, :, 0], codes[page, 1, :, 0] = 0x38, every
    s8[page, 1, :, 0] = scales[:, None]
    cache = runner.Kv8Cache(torch.from_numpy(codes).view(torch.float8_e4m3fn).cuda(), torch.from_numpy(s8).cuda())
    fn = runner.decode_kv8 if kind == "decode" else runner.prefill_kv8
    o, lse = fn(runner.DeviceBatch.from_host(b, kv_data=torch.empty(0)), cache)
    torch.cuda.synchronize()
    want = oracle.kv8_values(codes[page, 1, :, 0], s8[page, 1, :, 0])          # [requests, kv heads, dim]
    with np.errstate(over="ignore"):
        rounded = torch.from_numpy(want).to(torch.float32).to(dtype).float().numpy()
    np.testing.assert_array_equal(o.float().cpu().numpy(), np.repeat(rounded, 4, axis=1))
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("cap", [0.0, 6.0])
def test_prefill_with_and_without_split_tiles(dtype, g, cap):
    """Split tiles run on an instance of their own, with a merge."""
    for qo, kv, merges in (([40, 3], [3000, 700], True), ([30, 5], [100, 128], False)):
        b = batch(qo, kv, hq=2 * g, hkv=2, dtype=dtype, cap=cap, seed=g)
        cache, twin = quantised(b, 1)
        plan = runner.make_plan(b, api.PLAN_PREFILL_KV8)
        runner.plan_batch(plan, b)
        assert (plan.info().num_merge > 0) == merges
        o, lse = runner.prefill_kv8(runner.DeviceBatch.from_host(b, kv_data=torch.empty(0)), to_cuda(cache), plan)
        torch.cuda.synchronize()
        assert_attention(o, lse, twin, P_EPS["prefill"][dtype], f"merges {merges}")


@pytest.mark.parametrize("first", [0, 1])
def test_a_prefill_graph_replays_with_and_without_split_tiles(first):
    """Captured on a batch of one kind, replayed on both (the same total of rows, as the capture asks)."""
    bs = [batch([30, 5], [100, 128], seed=140, extra=0), batch([32, 3], [3000, 700], seed=141, extra=0)]
    pool = max(b.num_pages for b in bs)
    plan = api.Plan(api.PLAN_PREFILL_KV8, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, dtype=BF,
                    sm_scale=128 ** -0.5, max_batch=2, max_total_q=35, max_kv_pages=pool)
    cache = runner.Kv8Cache.zeros(pool, 2, 16, 128)
    s = torch.cuda.Stream()
    ix, ip, la, qo = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (pool, 3, 2, 3))
    q = torch.zeros(35, 8, 128, dtype=BF, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(35, 8, device="cuda")
    pairs = [quantised(b, 1, seed=i, poison=False) for i, b in enumerate(bs)]

    def load(i):
        b, (c, _) = bs[i], pairs[i]
        torch.cuda.synchronize()
        ix[:b.kv_indices.numel()].copy_(b.kv_indices)
        ip.copy_(b.kv_indptr), la.copy_(b.kv_last_page_len), qo.copy_(b.qo_indptr), q.copy_(b.q)
        cache.codes.view(torch.uint8)[:b.num_pages].copy_(c.codes.view(torch.uint8))
        cache.scales[:b.num_pages].copy_(c.scales)
        torch.cuda.synchronize()
        plan.plan(b.kv_indptr, b.kv_last_page_len, pool, qo_indptr_h=b.qo_indptr, kv_indices_h=b.kv_indices, stream=s)
        assert (plan.info().num_merge > 0) == (i == 1)

    step = lambda: plan.run(q, cache.codes, ix, ip, la, o, lse, qo_indptr=qo, kv_scales=cache.scales, stream=s)
    load(first)
    step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in (1 - first, first, 1 - first):
        load(i)
        o.fill_(99.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        assert_attention(o, lse, pairs[i][1], P_EPS["prefill"][BF], f"replay {i}")


@pytest.mark.parametrize("P", [1, 8, 16])
def test_decode_beside_a_bad_page_keeps_its_accuracy(P):
    b = batch([1] * 3, [40, 100, 64], P=P, seed=7)
    cache, twin = quantised(b)
    db = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0))
    plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
    runner.plan_batch(plan, b)
    db.kv_indices[int(b.kv_indptr[1])] = b.num_pages + 7     # request 1's first page
    o, lse = runner.decode_kv8(db, to_cuda(cache), plan)
    assert plan.device_error() == 1
    keep = [0, 2]
    ref_o, ref_lse = oracle.attention_of(twin, rows=keep)
    vmax = np.abs(np.nan_to_num(oracle.decode16(twin.kv_data)[:, 1])).max()
    got = oracle.decode16(o.cpu()[keep])
    assert (np.abs(got - ref_o) <= EPS2[BF] * np.abs(ref_o) + (2.0 ** -11 + 4e-4) * vmax).all()
    assert (np.abs(lse.cpu().numpy()[keep] - ref_lse) <= 4e-4).all()
