"""Which page tables the runner's eviction takes, without a GPU: what it refuses it refuses before any CUDA call."""
import dataclasses

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api, runner, workloads as W


def batch(shared=(), **kw):
    """Two requests of 40 and 30 keys in pages of 16 (3 and 2 of a pool of 9); shared: places of the list that hold
    the page of place 0."""
    b = W.make_paged_batch(qo_lens=[1, 1], kv_lens=[40, 30], num_qo_heads=2, num_kv_heads=1, head_dim=64, page_size=16,
                           dtype=torch.bfloat16, seed=1, pool_pages=9, identity_pages=True)
    ids = b.kv_indices.clone()
    for i in shared:
        ids[i] = ids[0]
    return type("HostOnly", (), {"host": dataclasses.replace(b, kv_indices=ids)})()


WEIGHTS = torch.zeros(9, 1, 16)


@pytest.mark.parametrize("shared", [[3], [1], [4, 3]])
def test_shared_pages_are_not_shortened_in_place(shared):
    with pytest.raises(ValueError, match="listed twice"):
        runner.evict(batch(shared), WEIGHTS, 20)


@pytest.mark.parametrize("pages,match", [([5, 6, 7], "4 pages"), ([[5, 6], [7, 8]], "4 pages"), ([5, 6, 7, 9], "of the pool"),
                                         ([-1, 6, 7, 8], "of the pool"), ([5, 6, 7, 7], "different"), ([5, 6, 7, 4], "different"),
                                         ([0, 6, 7, 8], "different")])
def test_pages_to_fill_are_free_ones_of_the_pool(pages, match):
    for shared in ([], [3]):
        if shared and 4 in pages:
            continue
        with pytest.raises(ValueError, match=match):
            runner.evict(batch(shared), WEIGHTS, 20, pages=pages)


@pytest.mark.parametrize("page", [-1, 9, 2 ** 31 - 1])
@pytest.mark.parametrize("pages", [None, [5, 6, 7, 8]])
def test_tables_past_the_pool_are_refused(page, pages):
    db = batch()
    db.host.kv_indices[1] = page
    with pytest.raises(ValueError, match="of the pool"):
        runner.evict(db, WEIGHTS, 20, pages=pages)


def evicted():
    db = batch()
    db.host = dataclasses.replace(db.host, moved=True)
    return db


def test_appends_by_slot_are_refused_after_an_eviction():
    """Keys and queries would be turned by their slots; without a rotation, or with positions, the call goes on (to
    the check of its tensors)."""
    rope, rows, cache = api.make_rope_axes(1e4, 64, [32]), torch.zeros(2, 1, 64, dtype=torch.bfloat16), runner.Kv8Cache(None, None)
    for call in (lambda: runner.append_kv(evicted(), rows, rows, rope_theta=1e4, rotate_q=False),
                 lambda: runner.append_kv_axes(evicted(), rows, rows, rope, rotate_q=False),
                 lambda: runner.append_kv8(evicted(), cache, rows, rows, rope, rotate_q=False)):
        with pytest.raises(ValueError, match="position"):
            call()
    for call in (lambda: runner.append_kv(batch(), rows, rows, rope_theta=1e4, rotate_q=False),
                 lambda: runner.append_kv(evicted(), rows, rows, rotate_q=False),
                 lambda: runner.append_kv_axes(evicted(), rows, rows, None, rotate_q=False),
                 lambda: runner.append_kv_axes(evicted(), rows, rows, rope, torch.zeros(1, 2, dtype=torch.int32), rotate_q=False)):
        with pytest.raises(AttributeError, match="qo_indptr"):   # past the check: the batch has no tensors on a GPU
            call()
