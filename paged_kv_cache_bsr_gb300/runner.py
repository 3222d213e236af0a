"""Run paged-KV attention on a workload through the C ABI (device marshalling only).

``DeviceBatch`` moves one paged batch to the GPU; ``decode``, ``prefill``,
``cascade`` and ``multi_level_cascade`` plan and launch through ``api.Plan`` and
return (o, lse) device tensors.  The arithmetic is all in libpkvbsr.so.

A call given a stream allocates what it makes on that stream, as torch does for work on
the current one: the outputs are good for the caller's current stream once that has
waited for it, and may be freed there at any time.  The caller's own tensors have to be
ready on the stream, and to outlive the call's work on it.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional, Sequence, Tuple, Union

import torch

from . import api


@dataclasses.dataclass
class DeviceBatch:
    host: object               # the workloads.PagedBatch it came from
    q: torch.Tensor
    kv_data: torch.Tensor
    qo_indptr: torch.Tensor
    kv_indptr: torch.Tensor
    kv_indices: torch.Tensor
    kv_last_page_len: torch.Tensor

    @staticmethod
    def from_host(b, device: str = "cuda", kv_data: Optional[torch.Tensor] = None) -> "DeviceBatch":
        to = lambda t: t.to(device, non_blocking=False).contiguous()
        return DeviceBatch(host=b, q=to(b.q), kv_data=to(b.kv_data) if kv_data is None else kv_data,
                           qo_indptr=to(b.qo_indptr), kv_indptr=to(b.kv_indptr), kv_indices=to(b.kv_indices),
                           kv_last_page_len=to(b.kv_last_page_len))


def _on(stream):
    """Allocations inside come from the pool of ``stream`` (None: the current one's).  Memory of another
    stream's pool could still be in use by that stream's earlier work, and a plan made for one call and
    dropped at its end be handed to that stream's next allocation while the call runs."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _handle(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _handle(stream) -> int:
    return stream if isinstance(stream, int) else stream.cuda_stream


def _returned(stream, *tensors):
    """Tensors made on ``stream``, kept from reuse until the caller's current stream is done with them too."""
    if stream is not None:
        now = torch.cuda.current_stream()
        if now.cuda_stream != _handle(stream):
            for t in tensors:
                t.record_stream(now)
    return tensors


def _limits_of(b, max_batch=None, max_total_q=None, max_kv_pages=None):
    return dict(max_batch=max_batch or max(b.batch, 1),
                max_total_q=max_total_q or max(b.total_q, 1),
                max_kv_pages=max_kv_pages or max(int(b.kv_indptr[-1]), 1))


def make_plan(b, kind: int, pipelined: bool = False, split_kv: bool = True, **limits) -> api.Plan:
    lim = _limits_of(b, **limits)
    return api.Plan(kind, num_qo_heads=b.num_qo_heads, num_kv_heads=b.num_kv_heads, head_dim=b.head_dim,
                    page_size=b.page_size, dtype=b.dtype, sm_scale=b.sm_scale, logits_cap=b.logits_cap,
                    causal=b.causal, pipelined=pipelined, split_kv=split_kv, **lim)


def plan_batch(plan: api.Plan, b, stream=None, num_pages: Optional[int] = None) -> None:
    """Plan the batch over a pool of ``num_pages`` pages (default: its own kv_data's)."""
    plan.plan(b.kv_indptr, b.kv_last_page_len, b.num_pages if num_pages is None else num_pages,
              qo_indptr_h=b.qo_indptr if plan.kind not in (api.PLAN_DECODE, api.PLAN_DECODE_KV8) else None,
              kv_indices_h=b.kv_indices, stream=stream)


def _outputs(q: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    return torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)


def decode(db: DeviceBatch, plan: Optional[api.Plan] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    b = db.host
    with _on(stream):
        if plan is None:
            plan = make_plan(b, api.PLAN_DECODE)
            plan_batch(plan, b, stream)
        o, lse = _outputs(db.q)
    plan.run(db.q, db.kv_data, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o, lse, stream=stream)
    return _returned(stream, o, lse)


def prefill(db: DeviceBatch, plan: Optional[api.Plan] = None, stream=None,
            mask: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Batch prefill; ``mask`` is an optional packed custom mask on the device
    (``workloads.pack_mask`` layout), applied on top of the batch's causal flag."""
    b = db.host
    with _on(stream):
        if plan is None:
            plan = make_plan(b, api.PLAN_PREFILL)
            plan_batch(plan, b, stream)
        o, lse = _outputs(db.q)
    plan.run(db.q, db.kv_data, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o, lse,
             qo_indptr=db.qo_indptr, mask=mask, stream=stream)
    return _returned(stream, o, lse)


def make_ragged_plan(q: torch.Tensor, k: torch.Tensor, qo_indptr, kv_indptr=None, sm_scale: Optional[float] = None,
                     logits_cap: float = 0.0, causal: bool = True, stream=None) -> api.Plan:
    """A plan for ``prefill_ragged`` over these tensors: qo_indptr and kv_indptr (None: the same) are the
    requests' rows of q and of k, on the host."""
    qo = torch.as_tensor(qo_indptr, dtype=torch.int32)
    kv = qo if kv_indptr is None else torch.as_tensor(kv_indptr, dtype=torch.int32)
    plan = api.Plan(api.PLAN_PREFILL_RAGGED, num_qo_heads=q.shape[1], num_kv_heads=k.shape[1], head_dim=q.shape[2],
                    page_size=1, dtype=q.dtype, sm_scale=q.shape[2] ** -0.5 if sm_scale is None else sm_scale,
                    logits_cap=logits_cap, causal=causal, max_batch=max(qo.numel() - 1, 1),
                    max_total_q=max(q.shape[0], 1), max_kv_pages=max(k.shape[0], 1))
    plan.plan(kv, None, k.shape[0], qo_indptr_h=qo, stream=stream)
    return plan


def prefill_ragged(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, qo_indptr=None, kv_indptr=None,
                   plan: Optional[api.Plan] = None, stream=None, **variant) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention over whole prompts before anything is in pages: q [total_q, Hq, d], k and v
    [total_kv, Hkv, d], the requests packed one behind another (views of a projection's output are
    read in place).  Without a plan one is made (``make_ragged_plan``, its arguments)."""
    with _on(stream):
        if plan is None:
            plan = make_ragged_plan(q, k, qo_indptr, kv_indptr, stream=stream, **variant)
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    plan.run_ragged(q, k, v, o, lse, stream=stream)
    return _returned(stream, o, lse)


def cascade(prefix: DeviceBatch, suffix: DeviceBatch, prefix_plan: Optional[api.Plan] = None,
            suffix_plan: Optional[api.Plan] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Shared-prefix attention: one prefill over the prefix row block (all
    requests' queries, no mask), one decode over the per-request suffixes, and
    merge_state of the two states, all on the GPU."""
    o_p, l_p = prefill(prefix, prefix_plan, stream)
    o_s, l_s = decode(suffix, suffix_plan, stream)
    api.merge_state(o_p, l_p, o_s, l_s, o_p, l_p, stream=stream)
    return o_p, l_p


def _positions_by_slot(b) -> None:
    if b.moved:
        raise ValueError("after an eviction a token's slot is not its position: give its position (append_kv_axes, append_kv8)")


def append_kv(db: DeviceBatch, k_new: torch.Tensor, v_new: torch.Tensor, rope_theta: float = 0.0,
              q_out: Optional[torch.Tensor] = None, rotate_q: bool = True, error: Optional[torch.Tensor] = None,
              stream=None) -> Optional[torch.Tensor]:
    """Append stage: write the batch's new tokens (one per query row, rows by
    qo_indptr) into ``db.kv_data`` at the end of each request's page list, turning
    the keys (and the queries, into ``q_out`` or a new tensor) by RoPE when
    rope_theta > 0 (by their slots: refused after ``evict``).  Returns the rotated queries (None with rotate_q
    False)."""
    b = db.host
    if rope_theta > 0:
        _positions_by_slot(b)
    params = api.make_params(b.num_qo_heads, b.num_kv_heads, b.head_dim, b.page_size, b.dtype, b.sm_scale)
    if rotate_q and q_out is None:
        with _on(stream):
            q_out = torch.empty_like(db.q)
        _returned(stream, q_out)
    api.append_paged_kv(params, db.qo_indptr, db.kv_indptr, db.kv_indices, db.kv_last_page_len, k_new, v_new,
                        db.kv_data, db.q if rotate_q else None, q_out if rotate_q else None, rope_theta,
                        error=error, stream=stream)
    return q_out if rotate_q else None


def append_kv_axes(db: DeviceBatch, k_new: torch.Tensor, v_new: torch.Tensor, rope: Optional[api.RopeAxes],
                   positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None, rotate_q: bool = True,
                   error: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """``append_kv`` with positions on several axes: ``rope`` from ``api.make_rope_axes`` (None: no
    rotation), ``positions`` [num_axes, new tokens] int32 on the device (None: each token's place in its
    request, refused after ``evict``).  Returns the rotated queries (None with rotate_q False)."""
    b = db.host
    if rope is not None and positions is None:
        _positions_by_slot(b)
    params = api.make_params(b.num_qo_heads, b.num_kv_heads, b.head_dim, b.page_size, b.dtype, b.sm_scale)
    if rotate_q and q_out is None:
        with _on(stream):
            q_out = torch.empty_like(db.q)
        _returned(stream, q_out)
    api.append_paged_kv_axes(params, rope, db.qo_indptr, db.kv_indptr, db.kv_indices, db.kv_last_page_len, positions,
                             k_new, v_new, db.kv_data, db.q if rotate_q else None, q_out if rotate_q else None,
                             error=error, stream=stream)
    return q_out if rotate_q else None


@dataclasses.dataclass
class Kv8Cache:
    """The 8-bit paged cache: e4m3 codes [num_pages, 2, Hkv, P, d] and one exponent byte per head
    row [num_pages, 2, Hkv, P] (a code c stands for e4m3(c) * 2^(byte - 127))."""

    codes: torch.Tensor
    scales: torch.Tensor

    @staticmethod
    def zeros(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, device: str = "cuda") -> "Kv8Cache":
        shape = (num_pages, 2, num_kv_heads, page_size)
        return Kv8Cache(torch.zeros(*shape, head_dim, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
                        torch.ones(shape, dtype=torch.uint8, device=device))

    @property
    def num_pages(self) -> int:
        return int(self.codes.shape[0])


def append_kv8(db: DeviceBatch, cache: Kv8Cache, k_new: torch.Tensor, v_new: torch.Tensor,
               rope: Optional[api.RopeAxes] = None, positions: Optional[torch.Tensor] = None,
               q_out: Optional[torch.Tensor] = None, rotate_q: bool = True, error: Optional[torch.Tensor] = None,
               stream=None) -> Optional[torch.Tensor]:
    """``append_kv_axes`` into the 8-bit cache (``db.kv_data`` is not used)."""
    b = db.host
    if rope is not None and positions is None:
        _positions_by_slot(b)
    params = api.make_params(b.num_qo_heads, b.num_kv_heads, b.head_dim, b.page_size, b.dtype, b.sm_scale)
    if rotate_q and q_out is None:
        with _on(stream):
            q_out = torch.empty_like(db.q)
        _returned(stream, q_out)
    api.append_paged_kv8(params, rope, db.qo_indptr, db.kv_indptr, db.kv_indices, db.kv_last_page_len, positions, k_new,
                         v_new, cache.codes, cache.scales, db.q if rotate_q else None, q_out if rotate_q else None,
                         error=error, stream=stream)
    return q_out if rotate_q else None


def _run_kv8(kind: int, db: DeviceBatch, cache: Kv8Cache, plan: Optional[api.Plan], stream
             ) -> Tuple[torch.Tensor, torch.Tensor]:
    with _on(stream):
        if plan is None:
            plan = make_plan(db.host, kind)
            plan_batch(plan, db.host, stream, num_pages=cache.num_pages)
        o, lse = _outputs(db.q)
    plan.run(db.q, cache.codes, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o, lse,
             qo_indptr=db.qo_indptr if kind == api.PLAN_PREFILL_KV8 else None, kv_scales=cache.scales, stream=stream)
    return _returned(stream, o, lse)


def decode_kv8(db: DeviceBatch, cache: Kv8Cache, plan: Optional[api.Plan] = None, stream=None
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """``decode`` over the 8-bit cache (a plan of kind PLAN_DECODE_KV8)."""
    return _run_kv8(api.PLAN_DECODE_KV8, db, cache, plan, stream)


def prefill_kv8(db: DeviceBatch, cache: Kv8Cache, plan: Optional[api.Plan] = None, stream=None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
    """``prefill`` over the 8-bit cache (a plan of kind PLAN_PREFILL_KV8)."""
    return _run_kv8(api.PLAN_PREFILL_KV8, db, cache, plan, stream)


def cascade_kv8(prefix: DeviceBatch, suffix: DeviceBatch, cache: Kv8Cache, prefix_plan: Optional[api.Plan] = None,
                suffix_plan: Optional[api.Plan] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``cascade`` over the 8-bit cache: the shared prefix once for all rows, then the suffixes, merged."""
    o_p, l_p = prefill_kv8(prefix, cache, prefix_plan, stream)
    o_s, l_s = decode_kv8(suffix, cache, suffix_plan, stream)
    api.merge_state(o_p, l_p, o_s, l_s, o_p, l_p, stream=stream)
    return o_p, l_p


def zero_key_weights(num_pages: int, num_kv_heads: int, page_size: int, device: str = "cuda") -> torch.Tensor:
    """Key weights beside a cache of that many pages, as long as it holds no key that was weighed."""
    return torch.zeros(num_pages, num_kv_heads, page_size, dtype=torch.float32, device=device)


def add_key_weights(db: DeviceBatch, lse: torch.Tensor, weights: torch.Tensor, cache: Optional[Kv8Cache] = None,
                    decay: float = 1.0, weighed_len: Optional[torch.Tensor] = None, error: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """Add to ``weights`` the probabilities that the batch's rows gave every key they see; ``lse`` from the
    attention call (or merged from several) over the same keys.  ``cache``: the keys of the 8-bit cache.  A page may
    be listed once.  A key's old weight is what its slot holds: 0 for a new key in a slot of ``zero_key_weights`` that
    held none, or behind what ``evict`` kept; where a page comes back by another way (a request that ended, a prefix
    that nothing lists any more), clear its weights, or give ``weighed_len`` [batch] int32, the keys of each request
    that have weights already."""
    b = db.host
    params = api.make_params(b.num_qo_heads, b.num_kv_heads, b.head_dim, b.page_size, b.dtype, b.sm_scale, b.logits_cap, b.causal)
    api.add_key_weights(params, db.kv_indptr, db.kv_indices, db.kv_last_page_len, db.q, lse,
                        db.kv_data if cache is None else cache.codes, weights, qo_indptr=None if b.is_decode else db.qo_indptr,
                        kv_scales=None if cache is None else cache.scales, decay=decay, weighed_len=weighed_len, error=error,
                        stream=stream)


def _pages_listed_once(ids: torch.Tensor, what: str) -> None:
    if ids.numel() and int(torch.bincount(ids).max()) > 1:
        raise ValueError(what)


def evict(db: DeviceBatch, weights: torch.Tensor, budget: Union[int, Sequence[int]], sink: int = 0, window: int = 0,
          cache: Optional[Kv8Cache] = None, error: Optional[torch.Tensor] = None, stream=None,
          pages: Union[None, Sequence[int], torch.Tensor] = None) -> Tuple[DeviceBatch, torch.Tensor]:
    """Shorten each request's cache to ``budget`` keys (one number, or one a request): for every kv head the last
    ``window``, the first ``sink`` and the heaviest others.  In place, which needs every page to be listed once (a
    batch with shared pages is refused, and no other batch may list them), or into ``pages``: ids of free pages of the
    pool on the host, of which the first ones are filled, for pages that requests share.
    Returns the batch with its shorter page tables, and the ids of the pages it no longer lists (on the host; with
    ``pages`` all it listed before, which other batches may still list).
    The key weights move with their keys, and are 0 in the kept pages' slots behind them and, in place, in the pages
    that are no longer listed, so that a key that comes to lie there starts from 0.  A new token's slot is no longer its
    position, so later appends need it given (``append_kv_axes``, ``append_kv8``; its count in the whole sequence), and
    those that would turn keys by their slots refuse the batch.  Nothing is read back from the GPU."""
    b = db.host
    budgets = [int(budget)] * b.batch if isinstance(budget, int) else [int(x) for x in budget]
    if len(budgets) != b.batch or min(budgets, default=0) < 0:
        raise ValueError("budget must be a count of keys, or one for each request")
    kept = [min(n, x) for n, x in zip(b.kv_lens, budgets)]
    used = [-(-n // b.page_size) for n in kept]
    indptr = torch.zeros(b.batch + 1, dtype=torch.int32)
    indptr[1:] = torch.tensor(used, dtype=torch.int32).cumsum(0)
    first = [int(x) for x in b.kv_indptr]
    source = b.kv_indices[first[0]:first[-1]]
    none = source[:0]
    if source.numel() and not 0 <= int(source.min()) <= int(source.max()) < weights.shape[0]:
        raise ValueError("kv_indices must be pages of the pool")
    if pages is None:
        _pages_listed_once(source, "a page is listed twice: shared pages need others to move their keys to (pages)")
        indices = torch.cat([none, *(b.kv_indices[s:s + n] for s, n in zip(first, used))])
        freed = torch.cat([none, *(b.kv_indices[s + n:e] for s, n, e in zip(first, used, first[1:]))])
    else:
        given = torch.as_tensor(pages, dtype=torch.int32).cpu()
        if given.dim() != 1 or given.numel() < int(indptr[-1]):
            raise ValueError("pages must be a list of %d pages" % int(indptr[-1]))
        indices, freed = given[:int(indptr[-1])].contiguous(), torch.unique(source)
        if indices.numel() and not 0 <= int(indices.min()) <= int(indices.max()) < weights.shape[0]:
            raise ValueError("pages must be pages of the pool")
        _pages_listed_once(torch.cat([indices, freed]), "pages must be different ones that the batch does not list")
    host = dataclasses.replace(b, kv_indptr=indptr, kv_indices=indices, kv_lens=kept, moved=b.moved or kept != list(b.kv_lens),
                               kv_last_page_len=torch.tensor([n - (p - 1) * b.page_size if n else 0 for n, p in zip(kept, used)],
                                                             dtype=torch.int32))
    with _on(stream):
        host_budget = torch.tensor(kept, dtype=torch.int32)  # (what they asked for may not fit 32 bits)
        keep = torch.empty(b.batch, b.num_kv_heads, max(kept, default=0), dtype=torch.int32, device=db.q.device)
        kept_len = torch.empty(b.batch, dtype=torch.int32, device=db.q.device)
        tables = [t.to(db.q.device) for t in (host.kv_indptr, host.kv_indices, host.kv_last_page_len)]
        api.select_keys(db.kv_indptr, db.kv_indices, db.kv_last_page_len, weights, host_budget.to(db.q.device), keep, kept_len,
                        sink=sink, window=window, error=error, stream=stream)
        api.compact_paged_kv(db.kv_indptr, db.kv_indices, db.kv_last_page_len, keep, kept_len,
                             db.kv_data if cache is None else cache.codes, kv_scales=None if cache is None else cache.scales,
                             weights=weights, dst_indptr=None if pages is None else tables[0],
                             dst_indices=None if pages is None else tables[1], error=error, stream=stream)
        # Slots that hold no key any more, and the last pages' behind the keys, weigh nothing.
        ends = [(int(indices[e - 1]), last) for e, n, last in zip(indptr[1:], used, host.kv_last_page_len) if 0 < n and last < b.page_size]
        if ends:
            at, last = (torch.tensor(x).to(db.q.device) for x in zip(*ends))
            behind = torch.arange(b.page_size, device=db.q.device) >= last.unsqueeze(1)
            weights[at] = weights[at].masked_fill(behind.unsqueeze(1), 0)
        if pages is None and freed.numel():
            weights.index_fill_(0, freed.to(db.q.device, torch.int64), 0)
    _returned(stream, *tables)
    return dataclasses.replace(db, host=host, kv_indptr=tables[0], kv_indices=tables[1], kv_last_page_len=tables[2]), freed


def mixed(db: DeviceBatch, plan: Optional[api.Plan] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """A batch mixing single-row (decode) and multi-row (prefill) requests in one
    call: the plan routes each request by its row count and splits the SMs, and one
    persistent launch runs both halves."""
    b = db.host
    with _on(stream):
        if plan is None:
            plan = make_plan(b, api.PLAN_MIXED)
            plan_batch(plan, b, stream)
        o, lse = _outputs(db.q)
    plan.run(db.q, db.kv_data, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o, lse,
             qo_indptr=db.qo_indptr, stream=stream)
    return _returned(stream, o, lse)


def levels_mixed(db: DeviceBatch, n_levels: int, plan: Optional[api.Plan] = None, stream=None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """A prefix tree (or a cascade, n_levels = 2) as one mixed launch: ``db`` holds
    ``workloads.levels_as_mixed(levels)``.  Multi-row nodes run on the prefill half
    of the mixed kernel and single-row nodes on its decode half; one n-state
    merge_state then folds every level's rows into the last level's."""
    o, lse = mixed(db, plan, stream)
    R = db.q.shape[0] // n_levels
    o_out, l_out = o[(n_levels - 1) * R:], lse[(n_levels - 1) * R:]
    # every level's states at once, into the last level's rows
    api.merge_states(o, lse, n_levels, o_out, l_out, stream=stream)
    return o_out, l_out


def cascade_mixed(db: DeviceBatch, plan: Optional[api.Plan] = None, stream=None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cascade attention as one mixed launch (``workloads.cascade_as_mixed``)."""
    return levels_mixed(db, 2, plan, stream)


def level_kind(b) -> int:
    """A level whose nodes each hold one query row is plain decode; a level with
    multi-row blocks (a prefix shared by several requests) runs on the prefill
    kernel without a mask, so each node's KV is read once for all its rows."""
    return api.PLAN_DECODE if all(n == 1 for n in b.qo_lens) else api.PLAN_PREFILL


def multi_level_cascade(levels: Sequence[DeviceBatch], plans: Optional[Sequence[api.Plan]] = None,
                        stream=None, side_streams: Optional[Sequence] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention over a prefix tree stored as one BSR matrix per level (greptalks
    summary, "Composable Formats for Shared Prefixes": one block-sparse matrix
    decomposed into several with different row-block sizes; fdeinterviews summary,
    "One format": shared prefixes as large row blocks, no data moved).

    Each level's batch groups the request rows into consecutive blocks (its nodes),
    each block against that node's pages; every level covers every row once.  Each
    level is computed on the GPU (prefill kernel for multi-row blocks, decode kernel
    for single rows) and the states are folded into level 0's buffers with
    merge_state.  With ``side_streams`` (one per level after the first) the levels
    run concurrently and join before the merges; the whole call is capturable in
    one CUDA graph.
    """
    if not levels:
        raise ValueError("multi_level_cascade needs at least one level")
    if plans is None:
        plans = []
        with _on(stream):
            for db in levels:
                p = make_plan(db.host, level_kind(db.host))
                plan_batch(p, db.host, stream)
                plans.append(p)
    if len(plans) != len(levels):
        raise ValueError("one plan per level")
    if side_streams is not None and len(side_streams) < len(levels) - 1:
        raise ValueError("one side stream per level after the first")
    q = levels[0].q
    with _on(stream):
        outs = [_outputs(q) for _ in levels]
    main = stream if stream is not None else torch.cuda.current_stream()

    def run(i, s):
        db, p = levels[i], plans[i]
        o, lse = outs[i]
        p.run(db.q, db.kv_data, db.kv_indices, db.kv_indptr, db.kv_last_page_len, o, lse,
              qo_indptr=db.qo_indptr if p.kind == api.PLAN_PREFILL else None, stream=s)

    if side_streams is None:
        for i in range(len(levels)):
            run(i, main)
    else:
        fork = torch.cuda.Event()
        fork.record(main)
        joins = []
        for i in range(1, len(levels)):
            s = side_streams[i - 1]
            s.wait_event(fork)
            run(i, s)
            ev = torch.cuda.Event()
            ev.record(s)
            joins.append(ev)
        run(0, main)
        for ev in joins:
            main.wait_event(ev)
    o0, l0 = outs[0]
    for o, lse in outs[1:]:
        api.merge_state(o0, l0, o, lse, o0, l0, stream=main)
    return _returned(stream, o0, l0)
