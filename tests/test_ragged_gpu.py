"""GPU parity of the prefill over packed keys and values (no pages) with plain attention in 64 bits."""
import math

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api, runner

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
EPS2 = {BF: 2.0 ** -8, FP: 2.0 ** -11}   # half a step, relative
LSE_OFF = 4e-4


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


def indptr(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def tensors(qo, kv, hq, hkv, dtype, seed=0, fused=False, gap=0):
    g = torch.Generator("cuda").manual_seed(seed)
    rows = lambda n, h: torch.randn(n, h, 128, generator=g, device="cuda").to(dtype)
    if fused:
        x = rows(sum(qo), hq + 2 * hkv + gap)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    return rows(sum(qo), hq), rows(sum(kv), hkv), rows(sum(kv), hkv)


def plain(q, k, v, qo, kv, causal, cap=0.0, sm_scale=None):
    """(o, lse, largest |value| that counts) in 64 bits."""
    sm = q.shape[2] ** -0.5 if sm_scale is None else sm_scale
    o, lse = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    vmax = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    g = q.shape[1] // k.shape[1]
    for (r0, r1), (k0, k1) in zip(zip(indptr(qo), indptr(qo)[1:]), zip(indptr(kv), indptr(kv)[1:])):
        kk, vv = (x[k0:k1].double().repeat_interleave(g, 1).transpose(0, 1) for x in (k, v))
        y = sm * torch.matmul(q[r0:r1].double().transpose(0, 1), kk.transpose(1, 2))
        if cap > 0:
            y = cap * torch.tanh(y / cap)
        if causal:
            y = y.masked_fill(torch.ones_like(y, dtype=torch.bool).triu(k1 - k0 - (r1 - r0) + 1), -math.inf)
        l = torch.logsumexp(y, -1)
        p = torch.exp(y - l.clamp(min=-1e300).unsqueeze(-1))
        o[r0:r1], lse[r0:r1] = torch.matmul(p, vv).transpose(0, 1), l.transpose(0, 1)
        vmax[r0:r1] = vv.abs().amax((1, 2)) if k1 > k0 else 0.0
    return o, lse, vmax


def check(o, lse, ref, dtype):
    """Logits are exact products summed in fp32, 128 terms of sum |q k| sm_scale ~ 10: off by less than 2e-4,
    a probability by that share (4e-4 with its exponential) and by half a 16-bit step, a weighted mean of
    values by that share of the largest, and the output by half a step of its own."""
    ro, rl, vmax = ref
    empty = torch.isneginf(rl)
    assert torch.equal(empty, torch.isneginf(lse))
    assert (lse.double() - rl)[~empty].abs().max() <= LSE_OFF if (~empty).any() else True
    bound = EPS2[dtype] * ro.abs() + (EPS2[dtype] + 4e-4) * vmax.unsqueeze(-1) + 2.0 ** -24
    off = (o.double() - ro).abs()
    assert bool((off <= bound).all()), float((off - bound).max())   # NaN fails too


@pytest.mark.parametrize("dtype,group,causal,cap,fused", [
    (BF, 4, True, 0.0, True), (FP, 4, True, 0.0, True), (BF, 1, True, 30.0, False), (FP, 2, False, 0.0, False),
    (BF, 8, True, 0.0, True), (FP, 8, False, 30.0, False), (BF, 2, True, 0.0, False), (FP, 1, False, 0.0, False)])
def test_matches_plain_attention(dtype, group, causal, cap, fused):
    """Lengths around the tile edges, one row, one key, more keys than rows and fewer, rows that see nothing."""
    qo = [1, 33, 128, 129, 300, 7, 0, 260]
    kv = qo if fused else [1, 40, 127, 500, 128, 3, 9, 257]
    q, k, v = tensors(qo, kv, 2 * group, 2, dtype, seed=group, fused=fused, gap=1)
    o, lse = runner.prefill_ragged(q, k, v, indptr(qo), indptr(kv), causal=causal, logits_cap=cap)
    check(o, lse, plain(q, k, v, qo, kv, causal, cap), dtype)


@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_few_rows_before_many_keys_split(hkv):
    """Tiles cut over their keys: the staged partial states and their merge."""
    qo, kv = [5, 64, 1], [5001, 3333, 130]
    q, k, v = tensors(qo, kv, 4 * hkv, hkv, BF, seed=hkv)
    plan = runner.make_ragged_plan(q, k, indptr(qo), indptr(kv))
    assert plan.info().num_merge > 0
    o, lse = runner.prefill_ragged(q, k, v, plan=plan)
    check(o, lse, plain(q, k, v, qo, kv, True), BF)


def test_requests_without_keys_and_batches_without_any():
    q, k, v = tensors([3, 2], [0, 4], 4, 2, FP)
    o, lse = runner.prefill_ragged(q, k, v, [0, 3, 5], [0, 0, 4], causal=False)
    assert torch.isneginf(lse[:3]).all() and not o[:3].any()
    check(o, lse, plain(q, k, v, [3, 2], [0, 4], False), FP)
    o, lse = runner.prefill_ragged(q, k[:0], v[:0], [0, 3, 5], [0, 0, 0])
    assert torch.isneginf(lse).all() and not o.any()
    o, lse = runner.prefill_ragged(q[:0], k, v, [0, 0], [0, 4])
    assert o.shape == (0, 4, 128)
    torch.cuda.synchronize()


def test_nothing_of_a_request_reaches_another():
    """NaN and infinite keys, values and queries of one request, and rows behind the last one."""
    qo, kv = [70, 50, 33], [70, 50, 33]
    q, k, v = tensors([*qo, 9], [*kv, 9], 8, 2, BF, seed=3)
    bad = slice(70, 120)
    for x in (q, k, v):
        x[bad] = float("nan")
        x[153:] = float("inf")
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    plan = api.Plan(api.PLAN_PREFILL_RAGGED, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=1, dtype=BF,
                    sm_scale=128 ** -0.5, causal=True, max_batch=3, max_total_q=153, max_kv_pages=153)
    plan.plan(torch.tensor(indptr(kv), dtype=torch.int32), None, 162, qo_indptr_h=torch.tensor(indptr(qo), dtype=torch.int32))
    plan.run_ragged(q[:153], k, v, o[:153], lse[:153])
    ref = plain(q, k, v, qo, kv, True)
    for part in (slice(0, 70), slice(120, 153)):
        check(o[part], lse[part], tuple(x[part] for x in ref), BF)
    assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
    assert (o[153:] == 7).all() and (lse[153:] == 7).all()
    assert plan.device_error() == 0


def test_a_key_that_is_nan_reaches_the_rows_that_see_it():
    q, k, v = tensors([200], [200], 4, 1, FP, seed=5)
    k[150] = float("nan")
    o, lse = runner.prefill_ragged(q, k, v, [0, 200])
    assert torch.isfinite(o[:150]).all() and torch.isnan(o[150:]).all() and torch.isnan(lse[150:]).all()


def test_strides_of_padded_rows_and_single_rows():
    q, k, v = tensors([1], [1], 8, 2, BF, seed=6, fused=True, gap=3)
    o, lse = runner.prefill_ragged(q, k, v, [0, 1])
    check(o, lse, plain(q, k, v, [1], [1], True), BF)
    big = torch.randn(40, 5, 3, 128, device="cuda").to(FP)
    k, v = big[:, 1, :2], big[:, 4, :2]
    q = torch.randn(40, 2, 128, device="cuda").to(FP)
    o, lse = runner.prefill_ragged(q, k, v, [0, 11, 40])
    check(o, lse, plain(q, k, v, [11, 29], [11, 29], True), FP)


def test_captured_and_replayed_with_another_batch():
    """A graph of the run call follows the plan: first without split tiles, then with them."""
    q, k, v = tensors([600], [600], 8, 2, BF, seed=7)
    plan = api.Plan(api.PLAN_PREFILL_RAGGED, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=1, dtype=BF,
                    sm_scale=128 ** -0.5, causal=True, max_batch=4, max_total_q=600, max_kv_pages=600)
    o, lse = torch.empty_like(q), torch.empty(600, 8, device="cuda")

    def use(lens):
        ip = torch.tensor(indptr(lens), dtype=torch.int32)
        plan.plan(ip, None, 600, qo_indptr_h=ip)

    use([600])
    plan.run_ragged(q, k, v, o, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run_ragged(q, k, v, o, lse)
    for lens in ([600], [1, 299, 300], [150, 150, 150, 150]):
        use(lens)
        graph.replay()
        check(o, lse, plain(q, k, v, lens, lens, True), BF)


def test_another_stream_and_equal_bits():
    q, k, v = tensors([300, 40], [300, 40], 8, 2, FP, seed=8, fused=True)
    a = runner.prefill_ragged(q, k, v, [0, 300, 340])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = runner.prefill_ragged(q, k, v, [0, 300, 340], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("lens", [(257, 64), (120, 128)])
def test_equals_the_paged_prefill(lens):
    """The same rows in pages: both within their error of the definition (the packed rows' keys are taken 64 at a
    time, the pages' 128, so the bits differ)."""
    n0, total = lens[0], sum(lens)
    q, k, v = tensors(lens, lens, 8, 2, BF, seed=9)
    rag = runner.make_ragged_plan(q, k, [0, n0, total])
    o, lse = runner.prefill_ragged(q, k, v, plan=rag)
    P, pages = 16, [-(-n // 16) for n in lens]
    kv = torch.zeros(sum(pages), 2, 2, P, 128, dtype=BF, device="cuda")
    for p0, r0, n in ((0, 0, n0), (pages[0], n0, lens[1])):
        i = torch.arange(n, device="cuda")
        kv[p0 + i // P, 0, :, i % P], kv[p0 + i // P, 1, :, i % P] = k[r0:r0 + n], v[r0:r0 + n]
    plan = api.Plan(api.PLAN_PREFILL, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=P, dtype=BF,
                    sm_scale=128 ** -0.5, causal=True, max_batch=2, max_total_q=total, max_kv_pages=sum(pages))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32)
    indptr_h, last_h = ints(0, pages[0], sum(pages)), ints(*(n - (p - 1) * P for n, p in zip(lens, pages)))
    plan.plan(indptr_h, last_h, sum(pages), qo_indptr_h=ints(0, n0, total))
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    plan.run(q, kv, torch.arange(sum(pages), dtype=torch.int32, device="cuda"), indptr_h.cuda(), last_h.cuda(), o2, lse2,
             qo_indptr=ints(0, n0, total).cuda())
    ref = plain(q, k, v, lens, lens, True)
    check(o, lse, ref, BF)
    check(o2, lse2, ref, BF)


@pytest.mark.parametrize("group,hkv,dtype,cap", [(4, 8, BF, 0.0), (1, 4, FP, 0.0), (8, 2, FP, 50.0)])
def test_a_maximum_that_grows_with_every_block(group, hkv, dtype, cap):
    """Logits that grow by 8 every 64 keys, so that every block's rows are summed against a new maximum, over many
    tiles of odd and even numbers of blocks a CTA.  (Their products' terms sum to less than 30: 128 x 30 x 2^-24 is
    2.3e-4, which with the cap's 43 x 2^-22 is within the 4e-4 that a logit may be off.)"""
    lens = [200, 33, 129, 70, 1, 190, 64, 65] * 4
    q, k, v = tensors(lens, lens, group * hkv, hkv, dtype, seed=group)
    u = torch.randn(128, generator=torch.Generator("cuda").manual_seed(1), device="cuda").sign()
    place = torch.cat([torch.arange(n, device="cuda") for n in lens]).view(-1, 1, 1)
    q = (u + 0.05 * q.float()).to(dtype)
    k = (u * place / 64 * (8 / 128 ** 0.5) + 0.05 * k.float()).to(dtype)
    o, lse = runner.prefill_ragged(q, k, v, indptr(lens), logits_cap=cap)
    check(o, lse, plain(q, k, v, lens, lens, True, cap), dtype)
