"""Refusals of the 8-bit cache's and the multi-axis appends' entry points (every check that comes before the
first CUDA call), their plans, and pins of the oracle's functions for them."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_bsr_gb300 import api, workloads as W

INVALID, UNSUPPORTED = -1, -3


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    oracle.build()
    return api.load()


@pytest.fixture(scope="module")
def ptrs():
    buf = torch.zeros(4096, dtype=torch.uint8)
    base = buf.data_ptr() + (-buf.data_ptr()) % 256
    return buf, ctypes.c_void_p(base), ctypes.c_void_p(base + 2)


# --------------------------------------------------------------------------- the oracle's functions
def test_e4m3_values_are_torchs():
    torch_v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    np.testing.assert_array_equal(oracle.e4m3_values(), torch_v)


def test_e4m3_round_is_torchs_and_goes_to_even():
    x = np.concatenate([np.random.default_rng(0).normal(size=20000) * 100, np.linspace(-448, 448, 7169),
                        2.0 ** -10 * np.arange(-40, 40)])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(oracle.e4m3_round(x), want)
    np.testing.assert_array_equal(oracle.e4m3_round([1.0625, 1.1875, 500.0, -np.inf]), [1.0, 1.25, 448.0, -448.0])


def test_kv8_exponents():
    x = np.array([[0.0, 0], [1.0, -1.5], [2.0, 0], [255.9, 1], [256, 1], [np.inf, 4], [2.0 ** -130, 0], [np.nan, -0.25]])
    np.testing.assert_array_equal(oracle.kv8_exponents(x), [1, 120, 121, 127, 128, 122, 1, 118])
    s = oracle.kv8_exponents(x)[[1, 2, 3, 4]]
    top = np.abs(x[[1, 2, 3, 4]]).max(-1) * 2.0 ** (127.0 - s)
    assert (top >= 128).all() and (top < 256).all()
    np.testing.assert_array_equal(oracle.kv8_values([[0x38, 0xB8]], [130]), [[8.0, -8.0]])


def test_rope_axes_with_equal_positions_is_rope():
    x, pos = np.random.default_rng(1).normal(size=(5, 3, 16)), np.array([0, 1, 7, -3, 1000])
    for inter in (False, True):
        got = oracle.rope_axes(x, np.tile(pos, (3, 1)), 1e4, 16, [3, 1, 4], inter)
        np.testing.assert_allclose(got, oracle.rope(x, pos, 1e4), atol=1e-12)


def test_rope_axes_deals_the_pairs():
    """Which axis turns which pair: unit vectors, one axis moved at a time."""
    sections, half = [3, 1, 2], 6
    want = {False: [0, 0, 0, 1, 2, 2], True: [0, 1, 2, 0, 2, 0]}
    for inter, axes in want.items():
        for i in range(half):
            x = np.zeros((3, 1, 16))
            x[:, 0, i] = 1.0
            y = oracle.rope_axes(x, np.eye(3) * 2, 100.0, 12, sections, inter)   # token a: position 2 on axis a
            moved = [bool(abs(y[a, 0, i] - 1) > 1e-9) for a in range(3)]
            assert moved == [a == axes[i] for a in range(3)]
            ang = 2 * 100.0 ** (-2 * i / 12)
            np.testing.assert_allclose([y[axes[i], 0, i], y[axes[i], 0, i + half]], [np.cos(ang), np.sin(ang)], atol=1e-12)
    x = np.random.default_rng(2).normal(size=(3, 2, 16))
    np.testing.assert_array_equal(oracle.rope_axes(x, np.eye(3), 100.0, 12, sections, False)[..., 12:], x[..., 12:])


# --------------------------------------------------------------------------- refusals
def rope(theta=1e4, rotary=128, sections=(16, 24, 24), axes=None, inter=0):
    r = api.RopeAxes(theta, rotary, len(sections) if axes is None else axes, (ctypes.c_int * 4)(*sections), inter)
    return r


@pytest.mark.parametrize("kv8", [False, True])
def test_appends_refuse_bad_arguments_before_any_cuda_call(lib, ptrs, kv8):
    _, p16, odd = ptrs
    good = api.make_params(8, 2, 128, 16, torch.bfloat16, 0.1)
    fn = lib.pkv_append_paged_kv8 if kv8 else lib.pkv_append_paged_kv_axes

    def append(params=good, r=rope(), batch=2, nnz=5, num_pages=10, k=p16, kv=p16, scales=p16, q_in=None, q_out=None,
               table=p16, positions=p16):
        args = [ctypes.byref(params) if params is not None else None, ctypes.byref(r) if r is not None else None, batch,
                nnz, num_pages, table, p16, p16, p16, positions, k, p16, kv]
        return fn(*args, *([scales] if kv8 else []), q_in, q_out, None, None)

    assert append(params=None) == INVALID
    for theta in (0.0, -1.0, float("nan"), float("inf"), 1e-30, 1e-308, 5e-324):
        assert append(r=rope(theta=theta)) == INVALID
    assert append(nnz=0, r=rope(theta=1e-9)) == api.PKV_OK
    for rotary, sections in ((0, (0,)), (8, (4,)), (24, (12,)), (144, (72,)), (128, (63,)), (128, (65, -1)), (128, (32, 32, 32))):
        assert append(r=rope(rotary=rotary, sections=sections)) == INVALID
    assert append(r=rope(axes=0)) == INVALID
    assert append(r=rope(axes=5)) == INVALID
    assert append(params=api.make_params(8, 2, 64, 16, torch.bfloat16, 0.1), r=rope()) == INVALID   # 128 of 64 elements
    assert append(params=api.make_params(8, 2, 96, 16, torch.bfloat16, 0.1), r=None) == UNSUPPORTED
    assert append(params=api.make_params(8, 2, 128, 16, api.PKV_F32, 0.1)) == UNSUPPORTED
    assert append(params=api.make_params(8, 0, 128, 16, torch.bfloat16, 0.1)) == INVALID
    assert append(params=api.make_params(8, 2, 128, 0, torch.bfloat16, 0.1)) == INVALID
    assert append(batch=-1) == INVALID
    assert append(nnz=-1) == INVALID
    assert append(num_pages=-1) == INVALID
    assert append(nnz=0) == api.PKV_OK
    assert append(nnz=0, k=None, kv=None) == api.PKV_OK
    assert append(batch=0) == INVALID
    assert append(nnz=1 << 31) == INVALID
    assert append(k=None) == INVALID
    assert append(k=odd) == INVALID
    assert append(kv=odd) == INVALID
    assert append(table=odd) == INVALID
    assert append(positions=odd) == INVALID
    assert append(q_in=p16) == INVALID
    assert append(q_out=p16) == INVALID
    assert append(q_in=p16, q_out=odd) == INVALID
    if kv8:
        assert append(scales=None) == INVALID
        assert append(scales=odd) == INVALID


def make(kind, params, lim=None, sms=152):
    return api.plan_create_host(kind, params, lim or api.Limits(4, 64, 1000), sms)


def test_run_calls_take_their_own_kinds_of_plan(lib, ptrs):
    _, p16, odd = ptrs
    b = W.mixed_batch(seed=6, n_decode=3, n_prefill=1)
    plans = {}
    for k in range(5):
        params = api.make_params(b.num_qo_heads, b.num_kv_heads, b.head_dim, b.page_size, b.dtype, b.sm_scale)
        h = api.plan_create_host(k, params, api.Limits(b.batch, b.total_q, int(b.kv_indptr[-1])), 152)
        _, host = api.plan_workspace_bytes(h)
        raw = torch.zeros(host + 64, dtype=torch.uint8)
        ws = raw[(-raw.data_ptr()) % 64:][:host]
        qo = b.qo_indptr if k not in (api.PLAN_DECODE, api.PLAN_DECODE_KV8) else None
        api.plan_compute(h, b.batch, qo, b.kv_indptr, b.kv_indices, b.kv_last_page_len, b.num_pages, ws)
        plans[k] = h
    runs = {
        "decode": lambda h: lib.pkv_batch_decode_paged(h, p16, p16, p16, p16, p16, p16, p16, p16, None),
        "prefill": lambda h: lib.pkv_batch_prefill_paged(h, *[p16] * 9, None),
        "masked": lambda h: lib.pkv_batch_prefill_paged_masked(h, *[p16] * 7, 1 << 40, p16, p16, p16, None),
        "mixed": lambda h: lib.pkv_batch_mixed_paged(h, *[p16] * 9, None),
        "noalloc": lambda h: lib.pkv_batch_decode_paged_noalloc(h, p16, 1 << 40, *[p16] * 7, None),
        "decode8": lambda h: lib.pkv_batch_decode_paged_kv8(h, *[p16] * 9, None),
        "prefill8": lambda h: lib.pkv_batch_prefill_paged_kv8(h, *[p16] * 10, None),
    }
    for name, run in runs.items():
        for k, h in plans.items():   # host-only plans: refused at the kind, or at the device check
            assert run(h) == INVALID, (name, k)
        assert run(None) == INVALID
    d8 = plans[api.PLAN_DECODE_KV8]
    for bad in range(9):
        if bad == 7:
            continue   # lse may be NULL
        args = [p16] * 9
        args[bad] = None
        assert lib.pkv_batch_decode_paged_kv8(d8, *args, None) == INVALID
    for h in plans.values():
        api.plan_destroy(h)


def test_kv8_plans(lib):
    """Decode over the 8-bit cache keeps decode tables for every group; prefill takes every page size and
    holds room for the expanded copy."""
    g8 = api.make_params(64, 8, 128, 16, torch.bfloat16, 0.1)
    lim = api.Limits(4, 4, 4096)
    a, c = make(api.PLAN_DECODE_KV8, g8, lim), make(api.PLAN_DECODE, g8, lim)
    assert api.plan_get_info(a).workers == 152 * 8 and api.plan_get_info(c).workers == 152
    assert lib.pkv_plan_set_split_kv(a, 0) == api.PKV_OK
    for h in (a, c):
        api.plan_destroy(h)
    for P in (1, 3, 16, 48):
        params = api.make_params(8, 2, 128, P, torch.bfloat16, 0.1)
        h = make(api.PLAN_PREFILL_KV8, params, api.Limits(4, 64, 1000))
        dev, _ = api.plan_workspace_bytes(h)
        assert dev >= (1000 * P + 15) // 16 * 2 * 2 * 16 * 128 * 2
        api.plan_destroy(h)
    for kind, params, st in [(api.PLAN_PREFILL_KV8, api.make_params(8, 2, 64, 16, torch.bfloat16, 0.1), UNSUPPORTED),
                             (api.PLAN_DECODE_KV8, api.make_params(8, 2, 128, 24, torch.bfloat16, 0.1), UNSUPPORTED),
                             (api.PLAN_DECODE_KV8, api.make_params(48, 2, 128, 16, torch.bfloat16, 0.1), UNSUPPORTED),
                             (api.PLAN_PREFILL_KV8, api.make_params(8, 2, 128, 16, api.PKV_F32, 0.1), UNSUPPORTED),
                             (5, api.make_params(8, 2, 128, 16, torch.bfloat16, 0.1), INVALID)]:
        with pytest.raises(api.PkvError) as e:
            make(kind, params)
        assert e.value.status == st


def test_the_binding_refuses_tensors_that_do_not_fit(lib):
    params, r = api.make_params(8, 2, 128, 16, torch.bfloat16, 0.1), api.make_rope_axes(1e4, 128, [16, 24, 24])
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    rows = lambda n, h, d=128, dt=torch.bfloat16: torch.zeros(n, h, d, dtype=dt)

    def call(ap=i(3), ip=i(3), ix=i(4), la=i(2), pos=torch.zeros(3, 5, dtype=torch.int32), k=rows(5, 2), v=rows(5, 2),
             kv8=torch.zeros(4, 2, 2, 16, 128, dtype=torch.uint8), sc=torch.zeros(4, 2, 2, 16, dtype=torch.uint8),
             q=rows(5, 8), q_out=None, rope_=r):
        with pytest.raises(ValueError):
            api.append_paged_kv8(params, rope_, ap, ip, ix, la, pos, k, v, kv8, sc, q, q_out)

    call()                                                     # host tensors
    call(ap=i(4))
    call(ip=torch.zeros(3, dtype=torch.int64))
    call(la=i(3))
    call(pos=torch.zeros(2, 5, dtype=torch.int32))
    call(pos=torch.zeros(3, 5))
    call(rope_=None)                                           # positions without a rotation
    call(k=rows(5, 2, dt=torch.float16))
    call(v=rows(4, 2))
    call(q_out=rows(5, 8, 64))
    call(kv8=torch.zeros(4, 2, 2, 16, 128, dtype=torch.bfloat16))
    call(sc=torch.zeros(4, 2, 2, 8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        api.append_paged_kv_axes(params, r, i(3), i(3), i(4), i(2), None, rows(5, 2), rows(5, 2), torch.zeros(4, 2, 2, 16, 128))
    with pytest.raises(ValueError):
        api.make_rope_axes(1e4, 128, [1, 2, 3, 4, 5])


# --------------------------------------------------------------------------- decode plans with the heads in step
def table(kv_lens, P):
    counts = [(n + P - 1) // P for n in kv_lens]
    indptr = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    last = torch.tensor([n - (c - 1) * P if c else 0 for n, c in zip(kv_lens, counts)], dtype=torch.int32)
    return counts, indptr, last


@pytest.mark.parametrize("hkv", [1, 2, 3, 5, 8, 16, 100, 700])
@pytest.mark.parametrize("P,seed", [(1, 0), (16, 1), (5, 2), (64, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_kv8_plan(lib, hkv, P, seed, d):
    gen = np.random.default_rng(seed)
    top = 1200 if hkv <= 16 else 40
    kv_lens = [0, 1] + [int(x) for x in gen.integers(1, top, size=20)] + [8 * top, 0, P, 17]
    counts, indptr, last = table(kv_lens, P)
    B = len(kv_lens)
    params = api.make_params(2 * hkv, hkv, d, P, torch.bfloat16, 0.1)
    h = make(api.PLAN_DECODE_KV8, params, api.Limits(B, B, int(indptr[-1])))
    _, host = api.plan_workspace_bytes(h)
    raw = torch.zeros(host + 64, dtype=torch.uint8)
    ws = raw[(-raw.data_ptr()) % 64:][:host]
    api.plan_compute(h, B, None, indptr, None, last, int(indptr[-1]) + 1, ws)
    info, work = api.plan_get_info(h), api.plan_get_work(h).tolist()
    W = info.workers
    assert W == 152 * (16 if d == 64 else 8)
    covered, slots, empty, load = set(), set(), {}, {}
    for w, b, kvh, p0, n, rows, slot, _ in work:
        assert 0 <= w < W and 0 <= kvh < hkv
        for p in range(p0, p0 + n):
            assert (b, kvh, p) not in covered
            covered.add((b, kvh, p))
        load[w] = load.get(w, 0) + n
        if n:
            assert rows == (int(last[b]) if p0 + n == counts[b] else P)
        else:
            empty[b] = empty.get(b, 0) + 1
        if slot >= 0:
            assert slot not in slots
            slots.add(slot)
    assert len(covered) == sum(counts) * hkv
    assert empty == {b: hkv for b, c in enumerate(counts) if c == 0}
    assert len(slots) == info.num_slots and slots == set(range(info.num_slots))
    assert [r[0] for r in work] == sorted(r[0] for r in work)
    # the slots of one (request, head) are neighbours in page order: the merge reads them as one range
    by = {}
    for w, b, kvh, p0, n, rows, slot, _ in work:
        if slot >= 0:
            by.setdefault((b, kvh), []).append((p0, slot))
    for pieces in by.values():
        s = [x for _, x in sorted(pieces)]
        assert len(s) > 1 and s == list(range(s[0], s[0] + len(s)))
    assert len(by) == info.num_merge
    if (W % hkv) * 20 <= W:
        # every head has the same pieces, a run's heads are neighbours (small pages: warps of one CTA where they
        # divide its warps), and no run is longer than its share
        cw = W // 152
        if P < 16 and cw % hkv == 0:
            ctas = {}
            for w, b, kvh, p0, n, _, _, _ in work:
                ctas.setdefault((b, p0), set()).add(w // cw)
            assert all(len(c) == 1 for c in ctas.values())
            run = lambda w: ((w % cw) // hkv * 152 + w // cw) * hkv + w % cw % hkv
        else:
            run = lambda w: (w % cw) * 152 + w // cw
        cuts = [{(b, p0, n) for _, b, kvh, p0, n, _, _, _ in work if kvh == x} for x in range(hkv)]
        assert all(c == cuts[0] for c in cuts)
        at = {(b, p0, kvh): run(w) for w, b, kvh, p0, n, _, _, _ in work}
        assert all(r == at[(b, p0, 0)] + kvh and at[(b, p0, 0)] % hkv == 0 for (b, p0, kvh), r in at.items())
        G = W // hkv
        T = max(16, -(-(8 * sum(counts) + 8 * (B + G - 1)) // G))
        assert max(load.values()) <= -(-T // 8)
    api.plan_destroy(h)


@pytest.mark.parametrize("kv_lens,hkv,P,share", [([1, 200, 0, 250], 2, 16, 8), ([128] * 64, 8, 16, 2), ([100] * 100, 8, 16, 1),
                                                 ([500] * 19, 8, 1, 8), ([40] * 152, 1, 5, 8), ([3] * 300, 1, 1, 4)])
def test_decode_kv8_plan_shares_short_lists_within_a_cta(lib, kv_lens, hkv, P, share):
    counts, indptr, last = table(kv_lens, P)
    B = len(kv_lens)
    h = make(api.PLAN_DECODE_KV8, api.make_params(hkv, hkv, 128, P, torch.bfloat16, 0.1), api.Limits(B, B, int(indptr[-1])))
    _, host = api.plan_workspace_bytes(h)
    raw = torch.zeros(host + 64, dtype=torch.uint8)
    ws = raw[(-raw.data_ptr()) % 64:][:host]
    api.plan_compute(h, B, None, indptr, None, last, int(indptr[-1]) + 1, ws)
    info, work = api.plan_get_info(h), api.plan_get_work(h).tolist()
    assert info.num_merge == 0 and info.num_slots == 0
    lists = {}
    for w, b, kvh, p0, n, rows, slot, _ in work:
        lists.setdefault((b, kvh), []).append((w, p0, n, slot))
        if n:
            assert rows == (int(last[b]) if p0 + n == counts[b] else P)
    assert len({w for w, *_ in work}) == len(work) and len(lists) == B * hkv
    for (b, kvh), pieces in lists.items():
        parts = max(1, min(share, counts[b]))
        assert len(pieces) == parts
        w0 = pieces[0][0]
        assert w0 % share == 0 and [w for w, *_ in pieces] == list(range(w0, w0 + parts))     # neighbours in one CTA
        assert [p for _, p, _, _ in pieces] == [counts[b] * i // parts for i in range(parts)]
        assert sum(n for _, _, n, _ in pieces) == counts[b]
        assert {s for *_, s in pieces} == ({-2} if parts > 1 else {-1})
    api.plan_destroy(h)
