"""Shared helpers of the 8-bit cache tests: an 8-bit cache with its 16-bit twin (the same values,
exactly), and the error bounds of attention over it."""
import dataclasses

import numpy as np
import torch

import oracle
from paged_kv_cache_bsr_gb300 import runner, workloads as W

EPS2 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative


def quantised(b, spread=0, seed=0, poison=True):
    """(codes, scales, twin) of a batch's kv_data: rows scaled by 2^U[-spread, spread], rounded to the
    8-bit cache; `twin` is the batch with the values the cache stands for as kv_data, exact in its dtype.
    Unreferenced pages and the slots behind each last page's keys hold NaN codes and scale 255."""
    gen = np.random.default_rng(seed)
    x = oracle.decode16(torch.nan_to_num(b.kv_data.float(), 0.0, 0.0, 0.0).to(b.dtype))
    x = x * 2.0 ** gen.integers(-spread, spread + 1, size=x.shape[:-1])[..., None]
    s = oracle.kv8_exponents(x)
    v = oracle.e4m3_round(x * 2.0 ** (127.0 - s)[..., None])
    table = {float(t): c for c, t in reversed(list(enumerate(oracle.e4m3_values())))}
    codes = np.array([table[t] for t in np.unique(v)], dtype=np.uint8)[np.searchsorted(np.unique(v), v)]
    twin = torch.from_numpy(oracle.kv8_values(codes, s)).to(b.dtype)
    assert np.array_equal(oracle.decode16(twin), oracle.kv8_values(codes, s))   # exact in the 16-bit dtype
    scales = s.astype(np.uint8)
    if poison:
        held = np.zeros((b.num_pages, b.page_size), dtype=bool)
        for r in range(b.batch):
            pages = b.kv_indices[int(b.kv_indptr[r]):int(b.kv_indptr[r + 1])].numpy()
            held[pages] = True
            if len(pages):
                held[pages[-1], int(b.kv_last_page_len[r]):] = False
        bad = np.broadcast_to(~held[:, None, None, :], scales.shape)
        codes = np.where(bad[..., None], 0x7F, codes).astype(np.uint8)
        scales = np.where(bad, 255, scales).astype(np.uint8)
    cache = runner.Kv8Cache(torch.from_numpy(codes).view(torch.float8_e4m3fn), torch.from_numpy(scales))
    return cache, dataclasses.replace(b, kv_data=twin)


def to_cuda(cache):
    return runner.Kv8Cache(cache.codes.cuda(), cache.scales.cuda())


def assert_attention(o, lse, twin, p_eps, what=""):
    """Against the fp64 oracle on the twin.  A probability rounded to 16 bits is off by p_eps relative; the
    logits are exact products summed in fp32: 128 terms of sum |q k| sm_scale log2(e) ~ 10 put them off by
    at most 128 * 2^-23 * 10 < 2e-4, a probability by that share and the lse by 2e-4 (4e-4 with what the
    exponentials and the logarithm add).  An output is a weighted mean of values of at most vmax, so it is
    off by (p_eps + 4e-4) vmax, and by half a step of its own rounding."""
    ref_o, ref_lse = oracle.attention_of(twin)
    o = oracle.decode16(o.cpu())
    lse = lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(o).all(), f"{what}: non-finite output"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(empty, np.isneginf(lse)), f"{what}: rows that see nothing"
    dl = np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, ref_lse))
    assert dl.max(initial=0) <= 4e-4, f"{what}: lse off by {dl.max():.2e}"
    kv = oracle.decode16(twin.kv_data)
    vmax = np.zeros((twin.total_q, twin.num_kv_heads))
    for r in range(twin.batch):
        k = twin.kv_lens[r]
        if not k:
            continue
        pages = twin.kv_indices[int(twin.kv_indptr[r]):int(twin.kv_indptr[r + 1])].numpy()
        v = kv[pages, 1].transpose(1, 0, 2, 3).reshape(twin.num_kv_heads, -1, twin.head_dim)[:, :k]
        vmax[int(twin.qo_indptr[r]):int(twin.qo_indptr[r + 1])] = np.abs(v).max(axis=(1, 2))
    vmax = np.repeat(vmax, twin.num_qo_heads // twin.num_kv_heads, axis=1)[..., None]
    bound = EPS2[twin.dtype] * np.abs(ref_o) + (p_eps + 4e-4) * vmax + 2.0 ** -24
    excess = np.abs(o - ref_o) - bound
    assert excess.max(initial=0) <= 0, f"{what}: output off by {np.abs(o - ref_o).max():.3e}, bound passed by {excess.max():.2e}"


def batch(qo_lens, kv_lens, hq=8, hkv=2, d=128, P=16, dtype=torch.bfloat16, seed=0, causal=False, cap=0.0, extra=2):
    need = sum((n + P - 1) // P for n in kv_lens)
    return W.make_paged_batch(qo_lens=qo_lens, kv_lens=kv_lens, num_qo_heads=hq, num_kv_heads=hkv, head_dim=d,
                              page_size=P, dtype=dtype, seed=seed, causal=causal, logits_cap=cap, pool_pages=need + extra)
