"""GPU parity of the appends with rotary positions on several axes (16-bit and 8-bit cache) and of
attention over the 8-bit cache, against the fp64 oracle, through the C ABI."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_bsr_gb300 import api, runner, workloads as W
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


# --------------------------------------------------------------------------- appends
# Sine and cosine (Taylor remainders, an angle rounded to 2^-25 of an eighth of a turn, the float
# result), two products and a sum: a turned element is off by less than 2^-21 of its pair's length.
TURN = 2.0 ** -21


def case(qo, kv, sections, rotary=None, interleaved=False, theta=1e4, pos=None, seed=0, **kw):
    b = batch(qo, kv, seed=seed, **kw)
    rotary = b.head_dim if rotary is None else rotary
    k_new, v_new = W.new_kv_rows(b, seed=seed + 1)
    if pos is None:
        pos = np.random.default_rng(seed).integers(-50, 5000, size=(len(sections), b.total_q))
    pos = np.asarray(pos, dtype=np.int32).reshape(len(sections), b.total_q)
    return b, k_new, v_new, pos, dict(theta=theta, rotary_dim=rotary, sections=list(sections), interleaved=interleaved)


def turned(x, pos, rope):
    """(turned rows, bound of their error before they are rounded)."""
    ref = oracle.rope_axes(x, pos, **rope)
    xv, h = oracle.decode16(x), rope["rotary_dim"] // 2
    r = np.hypot(xv[..., :h], xv[..., h:2 * h])
    return ref, TURN * np.concatenate([r, r, np.zeros_like(xv[..., 2 * h:])], -1)


def check_rounded(got, ref, err, dtype):
    bound = EPS2[dtype] * np.abs(ref) + err * 1.01 + 2.0 ** -25
    assert (np.abs(got - ref) <= bound).all(), f"off by {np.abs(got - ref).max():.3e}"


def check_codes(codes, scales, x, ref, err):
    """Stored head rows against exact ones: the exponent bytes equal, every code the nearest e4m3 or next
    to a border by no more than the error of what was rounded."""
    s = oracle.kv8_exponents(x)
    np.testing.assert_array_equal(scales, s)
    mul = 2.0 ** (127.0 - s)[..., None]
    y, e = ref * mul, err * mul
    got = oracle.e4m3_values()[codes]
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.maximum(np.abs(y), np.abs(got)), 2.0 ** -6))), -6) - 3)
    assert (np.abs(got - y) <= step / 2 + e).all()
    exact = got == oracle.e4m3_round(y)
    assert exact.mean() > 0.9999 or (~exact).sum() <= 2


def places(b):
    _, _, page, slot = oracle.append_positions(b.qo_indptr, b.kv_indptr, b.kv_last_page_len, b.kv_indices, b.page_size)
    return page, slot


def run_append(kind, b, k_new, v_new, pos, rope, fill=None, in_place=False, rotate_q=True):
    db = runner.DeviceBatch.from_host(b)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = None if rope is None else api.make_rope_axes(**rope)
    p = None if pos is None else torch.from_numpy(pos).cuda()
    kw = dict(q_out=db.q if in_place else None, rotate_q=rotate_q, error=err)
    cache = None
    if kind == "kv8":
        cache = runner.Kv8Cache.zeros(b.num_pages, b.num_kv_heads, b.page_size, b.head_dim)
        cache.codes.view(torch.uint8).fill_(0x5A)
        cache.scales.fill_(77)
        q = runner.append_kv8(db, cache, k_new.cuda(), v_new.cuda(), r, p, **kw)
    else:
        q = runner.append_kv_axes(db, k_new.cuda(), v_new.cuda(), r, p, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return db, cache, q


def check_append(kind, b, k_new, v_new, pos, rope, **kw):
    db, cache, q = run_append(kind, b, k_new, v_new, pos, rope, **kw)
    page, slot = places(b)
    if pos is None and rope:   # each token's place, on every axis
        _, place, _, _ = oracle.append_positions(b.qo_indptr, b.kv_indptr, b.kv_last_page_len, b.kv_indices, b.page_size)
        pos = np.tile(place, (len(rope["sections"]), 1))
    exact = lambda x: (oracle.decode16(x), np.zeros(x.shape))
    k_ref, k_err = turned(k_new, pos, rope) if rope else exact(k_new)
    q_ref, q_err = turned(b.q, pos, rope) if rope else exact(b.q)
    v_ref, v_err = exact(v_new)
    if q is not None:
        check_rounded(oracle.decode16(q.cpu()), q_ref, q_err, b.dtype)
    written = np.zeros((b.num_pages, b.page_size), dtype=bool)
    written[page, slot] = True
    if kind == "kv8":
        codes, scales = cache.codes.view(torch.uint8).cpu().numpy(), cache.scales.cpu().numpy()
        check_codes(codes[page, 0, :, slot], scales[page, 0, :, slot], oracle.decode16(k_new), k_ref, k_err)
        check_codes(codes[page, 1, :, slot], scales[page, 1, :, slot], oracle.decode16(v_new), v_ref, v_err)
        rest = np.broadcast_to(~written[:, None, None, :], scales.shape)
        assert (codes[rest] == 0x5A).all() and (scales[rest] == 77).all()   # nothing else written
    else:
        got = oracle.decode16(db.kv_data.cpu())
        check_rounded(got[page, 0, :, slot], k_ref, k_err, b.dtype)
        np.testing.assert_array_equal(got[page, 1, :, slot], v_ref)
        raw, was = db.kv_data.cpu().view(torch.int16).numpy(), b.kv_data.view(torch.int16).numpy()
        rest = np.broadcast_to(~written[:, None, None, :, None], raw.shape)
        np.testing.assert_array_equal(raw[rest], was[rest])


SHAPES = [
    dict(qo=[1, 5, 0, 33, 1], kv=[1, 40, 9, 33, 300], sections=[16, 24, 24], hq=32, hkv=8),
    dict(qo=[4, 1, 70], kv=[20, 1, 71], sections=[24, 20, 20], interleaved=True, hq=8, hkv=2, dtype=FP, theta=5e6),
    dict(qo=[2, 3, 17], kv=[9, 3, 18], sections=[7, 9], rotary=32, hq=7, hkv=1, d=64, P=5, dtype=FP),
    dict(qo=[6, 1], kv=[6, 50], sections=[8], rotary=16, hq=3, hkv=3, d=64, P=1),
    dict(qo=[3, 30], kv=[64, 31], sections=[1, 0, 30, 17], rotary=96, interleaved=True, hq=16, hkv=2, P=64),
    dict(qo=[1], kv=[1], sections=[64], hq=1, hkv=1, P=7),
]


@pytest.mark.parametrize("kind", ["kv16", "kv8"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_with_axes(kind, shape):
    check_append(kind, *case(**SHAPES[shape], seed=10 * shape))


@pytest.mark.parametrize("kind", ["kv16", "kv8"])
def test_append_without_rotation_and_without_queries(kind):
    b, k, v, _, _ = case([3, 1, 20], [3, 17, 300], [64], seed=5)
    check_append(kind, b, k, v, None, None)
    check_append(kind, b, k, v, None, None, rotate_q=False)


@pytest.mark.parametrize("kind", ["kv16", "kv8"])
def test_append_positions_default_to_the_places(kind):
    b, k, v, _, rope = case([3, 1, 20], [3, 170, 30], [20, 44], seed=6, theta=5e5)
    check_append(kind, b, k, v, None, rope)


@pytest.mark.parametrize("kind", ["kv16", "kv8"])
def test_queries_turned_in_place(kind):
    check_append(kind, *case([4, 9], [20, 9], [16, 24, 24], seed=7), in_place=True)


@pytest.mark.parametrize("kind", ["kv16", "kv8"])
def test_positions_over_the_whole_int32_range(kind):
    pos = np.array([[0, -1, 1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, -123456789, 131071],
                    [2 ** 31 - 1, 7, -2 ** 31, 0, 999999937, -1, 2 ** 30, -2 ** 30]])
    check_append(kind, *case([8], [8], [32, 32], pos=pos, seed=8))
    check_append(kind, *case([8], [8], [32, 32], pos=pos, seed=9, theta=0.5, interleaved=True))   # angles over a turn a step


def test_many_tokens_and_many_requests():
    """Grids that loop over the tokens, and more requests than are staged in shared memory."""
    qo = [3] * 1500
    check_append("kv8", *case(qo, [5] * 1500, [16, 24, 24], hq=4, hkv=2, seed=11))
    check_append("kv16", *case([6000, 1], [6001, 40], [16, 24, 24], hq=32, hkv=8, seed=12))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_kv8_rows_of_every_magnitude(dtype):
    """Zero rows, the smallest and largest values of the type, one element among zeros, powers of two."""
    b, k, v, pos, rope = case([8], [8], [64], hq=2, hkv=1, dtype=dtype, seed=13)
    tiny, big = torch.finfo(dtype).smallest_normal, torch.finfo(dtype).max
    for x in (k, v):
        x[0], x[1], x[2] = 0, x[1] * tiny, 0
        x[2, 0, 5] = big
        x[3] = x[3].float().mul(big / 8).clamp(-big, big).to(dtype)
        x[4] = 2.0 ** torch.arange(128).remainder(12).to(dtype)
        x[5] = tiny / 4
    check_append("kv8", b, k, v, pos, rope)


def test_kv8_non_finite_elements():
    b, k, v, pos, _ = case([2], [2], [64], hq=2, hkv=1, seed=14)
    v[0, 0, 3], v[0, 0, 4], v[0, 0, 5] = float("inf"), float("-inf"), float("nan")
    v[1] = float("inf")
    db, cache, _ = run_append("kv8", b, k, v, None, None)
    page, slot = places(b)
    codes, scales = cache.codes.view(torch.uint8).cpu().numpy(), cache.scales.cpu().numpy()
    got, s = codes[page, 1, 0, slot], scales[page, 1, 0, slot]
    assert got[0, 3] == 0x7E and got[0, 4] == 0xFE and got[0, 5] & 0x7F == 0x7F
    x = oracle.decode16(v)
    assert s[0] == oracle.kv8_exponents(x)[0, 0] and s[1] == 1 and (got[1] == 0x7E).all()
    rest = np.ones(128, dtype=bool)
    rest[3:6] = False
    np.testing.assert_array_equal(oracle.e4m3_values()[got[0, rest]], oracle.e4m3_round(x[0, 0, rest] * 2.0 ** (127.0 - s[0])))


@pytest.mark.parametrize("kind", ["kv16", "kv8"])
def test_append_flags_what_the_device_arrays_name_wrongly(kind):
    b, k, v, pos, rope = case([2, 3, 4], [18, 40, 7], [16, 24, 24], seed=15)
    db = runner.DeviceBatch.from_host(b)
    ix, ap = db.kv_indices.clone(), torch.tensor([0, 2, 5, 9], dtype=torch.int32, device="cuda")
    ix[int(b.kv_indptr[1]) - 1] = b.num_pages          # request 0's last page (both its new tokens)
    last = db.kv_last_page_len.clone()
    last[2] = 17                                        # request 2: a last page longer than a page
    db2 = dataclasses.replace(db, kv_indices=ix, kv_last_page_len=last, qo_indptr=ap)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = runner.Kv8Cache.zeros(b.num_pages, 2, 16, 128)
    before = db.kv_data.clone()
    r, p = api.make_rope_axes(**rope), torch.from_numpy(pos).cuda()
    if kind == "kv8":
        runner.append_kv8(db2, cache, k.cuda(), v.cuda(), r, p, error=err)
    else:
        runner.append_kv_axes(db2, k.cuda(), v.cuda(), r, p, error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 1 | 16
    if kind == "kv8":
        changed = (cache.scales != 1).any(2).any(1)
    else:
        changed = (db.kv_data.view(torch.int16) != before.view(torch.int16)).any(-1).any(2).any(1)
    page, slot = places(b)
    want = torch.zeros_like(changed)
    want[torch.from_numpy(page[2:5]), torch.from_numpy(slot[2:5])] = True   # request 1's tokens alone
    assert torch.equal(changed, want)


def test_append_of_nothing():
    b = batch([0, 0], [5, 9])
    db = runner.DeviceBatch.from_host(b)
    none = torch.empty(0, 2, 128, dtype=BF, device="cuda")
    cache = runner.Kv8Cache.zeros(b.num_pages, 2, 16, 128)
    runner.append_kv8(db, cache, none, none, rotate_q=False)
    torch.cuda.synchronize()
    assert int(cache.scales.max()) == 1


# --------------------------------------------------------------------------- attention
def check_attention(b, spread=3, seed=0, plan=None):
    cache, twin = quantised(b, spread, seed)
    db = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0))
    fn, kind = (runner.decode_kv8, "decode") if b.is_decode and not b.causal else (runner.prefill_kv8, "prefill")
    o, lse = fn(db, to_cuda(cache))
    torch.cuda.synchronize()
    assert_attention(o, lse, twin, P_EPS[kind][b.dtype], kind)


@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_decode_groups_dims_types(g, d, dtype):
    lens = [1, 2, 15, 16, 17, 0, 33, 250, 1000]
    check_attention(batch([1] * len(lens), lens, hq=3 * g, hkv=3, d=d, dtype=dtype, seed=g), spread=2)


@pytest.mark.parametrize("P", [1, 2, 3, 4, 5, 7, 8, 11, 12, 15, 16, 32, 48, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_page_sizes(P, d):
    lens = [1, P, P + 1, 3 * P, 16, 31, 100, 777]
    check_attention(batch([1] * len(lens), lens, d=d, P=P, seed=P))


@pytest.mark.parametrize("P", [1, 16, 64])
def test_decode_soft_cap(P):
    check_attention(batch([1] * 5, [1, 40, 333, 16, 4000], hq=16, hkv=4, P=P, cap=5.0, seed=1), spread=1)


def test_decode_split_over_the_workers():
    b = batch([1, 1, 1], [40000, 3, 12345], hq=8, hkv=1, P=16, seed=2)
    plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
    runner.plan_batch(plan, b)
    assert plan.info().num_merge == 2
    check_attention(b)
    check_attention(batch([1], [30000], hq=2, hkv=2, d=64, P=1, dtype=FP, seed=3))


def test_decode_scales_far_apart():
    """Values and keys whose scales differ by up to 2^16 from token to token (fp16: 2^10)."""
    check_attention(batch([1] * 3, [50, 500, 2000], seed=4), spread=8)
    check_attention(batch([1] * 3, [50, 500, 2000], seed=5, dtype=FP), spread=5)


def test_decode_queries_of_every_size():
    b = batch([1] * 4, [100] * 4, hq=8, hkv=1, seed=6)
    b.q[0] *= 2.0 ** 40    # logits of ~2^40: one key takes all
    b.q[1] *= 2.0 ** -60   # every key alike
    b.q[2, 3] = 0
    cache, twin = quantised(b, 1)
    o, lse = runner.decode_kv8(runner.DeviceBatch.from_host(b, kv_data=torch.empty(0)), to_cuda(cache))
    ref_o, ref_lse = oracle.attention_of(twin)
    o, lse = oracle.decode16(o.cpu()), lse.cpu().numpy()
    vmax = np.abs(oracle.decode16(twin.kv_data)[:, 1]).max()
    assert (np.abs(o - ref_o) <= EPS2[BF] * np.abs(ref_o) + (2.0 ** -11 + 4e-4) * vmax).all()
    assert (np.abs(lse - ref_lse) <= 4e-4 + 2.0 ** -18 * np.abs(ref_lse)).all()


def test_decode_bad_page_is_flagged_and_the_rest_exact():
    for P in (1, 8, 16):
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
        assert (np.abs(oracle.decode16(o.cpu()[keep]) - ref_o) <= 2.0 ** -8 * np.abs(ref_o) + 0.05).all()


@pytest.mark.parametrize("dtype,g", [(BF, 4), (FP, 1), (BF, 8), (FP, 2)])
@pytest.mark.parametrize("causal", [False, True])
def test_prefill_types_groups(dtype, g, causal):
    check_attention(batch([1, 40, 3, 200, 2], [5, 40, 0, 333, 700], hq=2 * g, hkv=2, dtype=dtype, causal=causal, seed=g), spread=2)


@pytest.mark.parametrize("P", [1, 3, 5, 8, 16, 24 * 2, 128])
def test_prefill_page_sizes(P):
    check_attention(batch([70, 2, 129], [200, 131, 129], P=P, causal=True, seed=P))


def test_prefill_rows_that_see_nothing():
    check_attention(batch([20, 5], [7, 0], causal=True, seed=8))


def test_prefill_against_states_of_another_length_and_soft_cap():
    check_attention(batch([300, 1, 17], [64, 1500, 900], causal=False, cap=8.0, seed=9), spread=1)


def test_cascade_over_the_8bit_cache():
    cb = W.cascade_decode(seed=3, batch=9, prefix_len=512, suffix_lo=5, suffix_hi=60, num_qo_heads=8, num_kv_heads=2)
    cache, twin = quantised(cb.full, 2, poison=False)
    dev = to_cuda(cache)
    empty = torch.empty(0)
    o, lse = runner.cascade_kv8(runner.DeviceBatch.from_host(cb.prefix, kv_data=empty),
                                runner.DeviceBatch.from_host(cb.suffix, kv_data=empty), dev)
    torch.cuda.synchronize()
    # two states of the output's type are merged: two more roundings of values of at most vmax
    assert_attention(o, lse, twin, EPS2[BF] * 3, "cascade")


# --------------------------------------------------------------------------- a run of them together
def serving_reference(b, cache):
    """Attention of the batch (already turned queries) over what the cache holds."""
    vals = oracle.kv8_values(cache.codes.view(torch.uint8).cpu().numpy(), cache.scales.cpu().numpy())
    return dataclasses.replace(b, kv_data=torch.from_numpy(vals).to(b.dtype))


def test_prompt_then_steps():
    """Prompts with pictures appended and attended causally, then three decode steps, one cache throughout."""
    hq, hkv, P, sections = 8, 2, 16, [16, 24, 24]
    prompts, steps = [37, 130, 64, 1], 3
    final = [n + steps for n in prompts]
    full = batch([1] * 4, final, hq=hq, hkv=hkv, P=P, seed=20, extra=1)
    cache = runner.Kv8Cache.zeros(full.num_pages, hkv, P, 128)
    rope = api.make_rope_axes(5e5, 128, sections)
    gen = np.random.default_rng(3)
    state = None
    for step in range(steps + 1):
        kv = [n + step for n in prompts]
        qo = prompts if step == 0 else [1] * 4
        counts = [(n + P - 1) // P for n in kv]
        pages = [full.kv_indices[int(full.kv_indptr[r]):int(full.kv_indptr[r]) + counts[r]] for r in range(4)]
        b = batch(qo, kv, hq=hq, hkv=hkv, P=P, seed=30 + step, causal=step == 0, extra=30)
        b.kv_indices = torch.cat(pages)
        k_new, v_new = W.new_kv_rows(b, seed=40 + step)
        pos = gen.integers(0, 3000, size=(3, b.total_q)).astype(np.int32)
        db = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0))
        q = runner.append_kv8(db, cache, k_new.cuda(), v_new.cuda(), rope, torch.from_numpy(pos).cuda())
        db.q = q
        o, lse = (runner.prefill_kv8 if step == 0 else runner.decode_kv8)(db, cache)
        torch.cuda.synchronize()
        check_rounded(oracle.decode16(q.cpu()), *turned(b.q, pos, dict(theta=5e5, rotary_dim=128, sections=sections, interleaved=False)), BF)
        kind = "prefill" if step == 0 else "decode"
        assert_attention(o, lse, serving_reference(dataclasses.replace(b, q=q.cpu()), cache), P_EPS[kind][BF], f"step {step}")


def test_a_step_replays_in_a_cuda_graph_after_replanning():
    """Append and decode captured once; other lengths planned into the same plan, other contents, replayed."""
    lens = [[20, 300, 47], [33, 5, 800]]
    bs = [batch([1] * 3, n, hq=8, hkv=2, seed=50 + i, extra=80) for i, n in enumerate(lens)]
    n_pages = 90
    max_pages = 64
    caches = [runner.Kv8Cache.zeros(n_pages, 2, 16, 128) for _ in bs]
    plan = api.Plan(api.PLAN_DECODE_KV8, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, dtype=BF,
                    sm_scale=128 ** -0.5, max_batch=3, max_kv_pages=max_pages)
    rope = api.make_rope_axes(1e4, 128, [16, 24, 24])
    s = torch.cuda.Stream()
    ix = torch.zeros(max_pages, dtype=torch.int32, device="cuda")
    ip, la = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    ap = torch.arange(4, dtype=torch.int32, device="cuda")
    q, qr = (torch.zeros(3, 8, 128, dtype=BF, device="cuda") for _ in range(2))
    k, v = (torch.zeros(3, 2, 128, dtype=BF, device="cuda") for _ in range(2))
    pos = torch.zeros(3, 3, dtype=torch.int32, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(3, 8, device="cuda")
    cache = runner.Kv8Cache.zeros(n_pages, 2, 16, 128)
    params = api.make_params(8, 2, 128, 16, BF, 1.0)

    def load(i):
        b = bs[i]
        c, _ = quantised(b, 1, seed=i, poison=False)
        for t, x in ((ip, b.kv_indptr), (la, b.kv_last_page_len), (q, b.q)):
            t.copy_(x)
        ix[:b.kv_indices.numel()].copy_(b.kv_indices)
        cache.codes.view(torch.uint8)[:b.num_pages].copy_(c.codes.view(torch.uint8)[:n_pages])
        cache.scales[:b.num_pages].copy_(c.scales)
        kn, vn = W.new_kv_rows(b, seed=60 + i)
        k.copy_(kn)
        v.copy_(vn)
        pos.copy_(torch.randint(0, 900, (3, 3), generator=torch.Generator().manual_seed(i), dtype=torch.int32))
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            plan.plan(b.kv_indptr, b.kv_last_page_len, n_pages, kv_indices_h=b.kv_indices, stream=s)

    def step():
        api.append_paged_kv8(params, rope, ap, ip, ix, la, pos, k, v, cache.codes, cache.scales, q, qr, stream=s)
        plan.run(qr, cache.codes, ix, ip, la, o, lse, kv_scales=cache.scales, stream=s)

    n_pages = max(b.num_pages for b in bs)
    cache = runner.Kv8Cache.zeros(n_pages, 2, 16, 128)
    load(0)
    step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for i in (1, 0):
        load(i)
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        torch.cuda.synchronize()
        b = bs[i]
        view = runner.Kv8Cache(cache.codes.view(torch.uint8)[:b.num_pages].view(torch.float8_e4m3fn), cache.scales[:b.num_pages])
        assert_attention(o, lse, serving_reference(dataclasses.replace(b, q=qr.cpu()), view), 2.0 ** -11, f"replay {i}")
        assert plan.device_error(stream=s) == 0


def test_rows_behind_the_batch_stay():
    """Outputs of a bigger buffer: rows past the batch's are left as they were."""
    b = batch([1] * 3, [40, 100, 7], seed=70)
    cache, _ = quantised(b)
    db = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0))
    o, lse = torch.full((5, 8, 128), 9.0, dtype=BF, device="cuda"), torch.full((5, 8), 9.0, device="cuda")
    plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
    runner.plan_batch(plan, b)
    c = to_cuda(cache)
    plan.run(db.q, c.codes, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o[:3], lse[:3], kv_scales=c.scales)
    torch.cuda.synchronize()
    assert bool((o[3:] == 9).all()) and bool((lse[3:] == 9).all()) and not bool((o[:3] == 9).any())


def test_decode_in_pipelined_plans_and_without_split():
    b = batch([1] * 4, [500, 33, 1200, 9], seed=71)
    cache, twin = quantised(b)
    c, db = to_cuda(cache), runner.DeviceBatch.from_host(b, kv_data=torch.empty(0))
    for kw in (dict(pipelined=True), dict(split_kv=False)):
        plan = runner.make_plan(b, api.PLAN_DECODE_KV8, **kw)
        for _ in range(3):
            runner.plan_batch(plan, b)
            o, lse = runner.decode_kv8(db, c, plan)
        torch.cuda.synchronize()
        assert_attention(o, lse, twin, 2.0 ** -11, str(kw))


def test_the_full_serving_batch():
    """The Llama-3-8B-shaped decode batch over the 8-bit cache (sampled rows against the oracle)."""
    b = W.llama3_decode(seed=1001, batch=24)
    check_attention(b, spread=1)


def test_a_pool_past_4_gib():
    """Pages at the end of a pool of more than 2^32 bytes: append, decode and prefill there."""
    hq, hkv, P, D = 8, 8, 128, 128
    n_pages = 17000                                  # 4.46 GB of codes
    cache = runner.Kv8Cache.zeros(n_pages, hkv, P, D)
    assert cache.codes.numel() > 1 << 32
    b = batch([130, 40], [300, 40], hq=hq, hkv=hkv, P=P, seed=80, causal=True, extra=0)
    far = n_pages - b.num_pages
    k_new, v_new = W.new_kv_rows(b, seed=81)
    small, twin = quantised(b, 1, poison=False)
    cache.codes.view(torch.uint8)[far:].copy_(small.codes.view(torch.uint8))
    cache.scales[far:].copy_(small.scales)
    shifted = dataclasses.replace(b, kv_indices=b.kv_indices + far)
    db = runner.DeviceBatch.from_host(shifted, kv_data=torch.empty(0))
    rope = api.make_rope_axes(1e4, 128, [64])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    db.q = runner.append_kv8(db, cache, k_new.cuda(), v_new.cuda(), rope, error=err)
    o, lse = runner.prefill_kv8(db, cache)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and int(cache.codes.view(torch.uint8)[:far].max()) == 0
    tail = runner.Kv8Cache(cache.codes.view(torch.uint8)[far:].view(torch.float8_e4m3fn), cache.scales[far:])
    ref = serving_reference(dataclasses.replace(b, q=db.q.cpu()), tail)
    assert_attention(o, lse, ref, P_EPS["prefill"][BF], "prefill")
    d = dataclasses.replace(shifted, qo_indptr=torch.tensor([0, 1, 2], dtype=torch.int32), qo_lens=[1, 1], q=b.q[:2], causal=False)
    o, lse = runner.decode_kv8(runner.DeviceBatch.from_host(d, kv_data=torch.empty(0)), cache)
    torch.cuda.synchronize()
    assert_attention(o, lse, serving_reference(dataclasses.replace(d, kv_indices=b.kv_indices, kv_data=b.kv_data), tail),
                     2.0 ** -11, "decode")
    # the 16-bit append past 2^32 bytes
    pool = torch.zeros(9000, 2, hkv, P, D, dtype=BF, device="cuda")
    off = 9000 - b.num_pages
    db16 = dataclasses.replace(db, kv_data=pool, kv_indices=(b.kv_indices + off).cuda(), q=b.q.cuda())
    runner.append_kv_axes(db16, k_new.cuda(), v_new.cuda(), None, rotate_q=False)
    page, slot = places(b)
    torch.testing.assert_close(pool[off:][torch.from_numpy(page), 0, :, torch.from_numpy(slot)].cpu(), k_new, rtol=0, atol=0)
    assert float(pool[:off].abs().max()) == 0


def test_runs_refuse_tensors_that_do_not_fit_the_plan():
    b = batch([1] * 3, [40, 100, 7], seed=82)
    cache, _ = quantised(b)
    c, db = to_cuda(cache), runner.DeviceBatch.from_host(b, kv_data=torch.empty(0))
    plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
    runner.plan_batch(plan, b)
    o, lse = torch.zeros_like(db.q), torch.zeros(3, 8, device="cuda")
    good = dict(q=db.q, kv=c.codes, ix=db.kv_indices, ip=db.kv_indptr, la=db.kv_last_page_len, o=o, lse=lse, scales=c.scales)

    def run(**kw):
        a = {**good, **kw}
        plan.run(a["q"], a["kv"], a["ix"], a["ip"], a["la"], a["o"], a["lse"], kv_scales=a["scales"])

    for bad in (dict(scales=None), dict(q=db.q.half()), dict(q=db.q[:2]), dict(o=o[:, :4]), dict(lse=lse.half()),
                dict(lse=lse[:2]), dict(kv=c.codes[:-1]), dict(kv=c.codes[:5], scales=c.scales[:5]), dict(scales=c.scales.int()),
                dict(ix=db.kv_indices[:-1]), dict(ip=db.kv_indptr.long()), dict(la=db.kv_last_page_len[:2]),
                dict(q=db.q.cpu()), dict(o=torch.zeros(3, 16, 128, dtype=BF, device="cuda")[:, ::2]), dict(lse=lse.cpu())):
        with pytest.raises(ValueError):
            run(**bad)
    with pytest.raises(ValueError):
        plan.run(db.q, c.codes, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o, lse, kv_scales=c.scales,
                 mask=torch.zeros(4, dtype=torch.uint8, device="cuda"))
    run(lse=None)
    with pytest.raises(ValueError):   # the 16-bit cache's plan takes no scales
        runner.make_plan(b, api.PLAN_DECODE).run(db.q, c.codes, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o,
                                                 kv_scales=c.scales)
    torch.cuda.synchronize()


def test_two_streams_with_their_own_plans():
    """Two steps of different batches on two streams at once, each with its plan and workspace."""
    bs = [batch([1] * 8, list(np.random.default_rng(s).integers(1, 3000, size=8)), hq=16, hkv=4, seed=90 + s) for s in range(2)]
    pairs = [quantised(b, 1, seed=s) for s, b in enumerate(bs)]
    streams = [torch.cuda.Stream() for _ in bs]
    jobs = []
    for b, (cache, _), s in zip(bs, pairs, streams):
        plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
        runner.plan_batch(plan, b, stream=s)
        jobs.append((runner.DeviceBatch.from_host(b, kv_data=torch.empty(0)), to_cuda(cache), plan, s))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [runner.decode_kv8(db, c, plan, stream=s) for db, c, plan, s in jobs]
    torch.cuda.synchronize()
    for (o, lse), (_, twin) in zip(outs, pairs):
        assert_attention(o, lse, twin, 2.0 ** -11)


def test_the_same_call_twice_gives_the_same_bits():
    b = batch([1] * 6, [9000, 3, 700, 64, 2000, 1], hq=8, hkv=1, seed=95)
    cache, _ = quantised(b, 2)
    c, db = to_cuda(cache), runner.DeviceBatch.from_host(b, kv_data=torch.empty(0))
    plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
    runner.plan_batch(plan, b)
    first = runner.decode_kv8(db, c, plan)
    for _ in range(10):
        again = runner.decode_kv8(db, c, plan)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("g,d,dtype,cap", [(1, 128, BF, 0.0), (2, 64, FP, 4.0), (4, 128, FP, 0.0), (8, 64, BF, 0.0), (8, 128, BF, 6.0)])
def test_decode_lists_shared_within_a_cta(g, d, dtype, cap):
    lens = [1, 16, 17, 0, 33, 250, 128, 400, 2]
    b = batch([1] * len(lens), lens, hq=2 * g, hkv=2, d=d, dtype=dtype, cap=cap, seed=g)
    plan = runner.make_plan(b, api.PLAN_DECODE_KV8)
    runner.plan_batch(plan, b)
    assert plan.info().num_merge == 0 and (plan.work()[:, 6] == -2).any()
    check_attention(b, spread=1)


def test_a_graph_captured_without_splits_merges_after_replanning():
    """Captured on a batch whose lists are shared within CTAs (nothing to merge), replayed on one whose
    long lists are split over the card, and back."""
    lens = [[20, 300], [30000, 17]]
    bs = [batch([1, 1], n, hq=8, hkv=2, seed=110 + i, extra=0) for i, n in enumerate(lens)]
    pool = max(b.num_pages for b in bs)
    plan = api.Plan(api.PLAN_DECODE_KV8, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, dtype=BF,
                    sm_scale=128 ** -0.5, max_batch=2, max_kv_pages=pool)
    cache = runner.Kv8Cache.zeros(pool, 2, 16, 128)
    s = torch.cuda.Stream()
    ix, ip, la = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (pool, 3, 2))
    q = torch.zeros(2, 8, 128, dtype=BF, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(2, 8, device="cuda")
    twins = []
    for i, b in enumerate(bs):
        c, twin = quantised(b, 1, seed=i, poison=False)
        twins.append((c, twin))

    def load(i):
        b, (c, _) = bs[i], twins[i]
        torch.cuda.synchronize()
        ix[:b.kv_indices.numel()].copy_(b.kv_indices)
        ip.copy_(b.kv_indptr), la.copy_(b.kv_last_page_len), q.copy_(b.q)
        cache.codes.view(torch.uint8)[:b.num_pages].copy_(c.codes.view(torch.uint8))
        cache.scales[:b.num_pages].copy_(c.scales)
        torch.cuda.synchronize()
        plan.plan(b.kv_indptr, b.kv_last_page_len, pool, kv_indices_h=b.kv_indices, stream=s)
        return plan.info().num_merge

    step = lambda: plan.run(q, cache.codes, ix, ip, la, o, lse, kv_scales=cache.scales, stream=s)
    assert load(0) == 0
    step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in (1, 0, 1):
        assert (load(i) > 0) == (i == 1)
        o.fill_(99.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        assert_attention(o, lse, twins[i][1], 2.0 ** -11, f"replay {i}")


def test_prefill_bad_page_is_flagged_and_the_rest_exact():
    b = batch([20, 30, 5], [40, 100, 64], causal=True, seed=120)
    cache, twin = quantised(b)
    db = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0))
    plan = runner.make_plan(b, api.PLAN_PREFILL_KV8)
    runner.plan_batch(plan, b)
    db.kv_indices[int(b.kv_indptr[1])] = -3          # request 1's first page
    o, lse = runner.prefill_kv8(db, to_cuda(cache), plan)
    assert plan.device_error(clear=True) == 1 and plan.device_error() == 0
    keep = list(range(20)) + list(range(50, 55))
    ref_o, ref_lse = oracle.attention_of(twin, rows=keep)
    got = oracle.decode16(o.cpu()[keep])
    vmax = np.abs(np.nan_to_num(oracle.decode16(twin.kv_data)[:, 1])).max()
    assert (np.abs(got - ref_o) <= EPS2[BF] * np.abs(ref_o) + (EPS2[BF] + 4e-4) * vmax).all()
    assert (np.abs(lse.cpu().numpy()[keep] - ref_lse) <= 4e-4).all()


@pytest.mark.parametrize("hkv,d,P", [(40, 128, 16), (150, 64, 4), (700, 64, 16), (2500, 64, 1)])
def test_decode_many_kv_heads(hkv, d, P):
    """Plans with many heads in step, and (700 heads fill 152 x 16 workers badly, 2500 are more than them) list by list."""
    lens = [1, 33, 60, 7] if hkv > 200 else [1, 700, 33, 0, 1500, 64]
    check_attention(batch([1] * len(lens), lens, hq=hkv, hkv=hkv, d=d, P=P, seed=hkv), spread=1)
