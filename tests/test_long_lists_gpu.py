"""GPU tests of the choice and the move at the end of 32-bit counts."""
import pytest
import torch

from paged_kv_cache_bsr_gb300 import api
from length_util import BF, ints

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1 - 2 ** 21   # keys of a request


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


def table(keys, P):
    """A request that lists one page again and again."""
    pages = -(-keys // P)
    return ints([0, pages]), torch.zeros(pages, dtype=torch.int32, device="cuda"), ints([keys - (pages - 1) * P])


@pytest.mark.parametrize("P", [1008, 2 ** 20])
def test_requests_past_the_most_keys_keep_and_move_nothing(P):
    w, keep, kept, kv = torch.rand(1, 1, P, device="cuda"), ints([[[0, 1, 2]]]), ints([5]), torch.zeros(1, 2, 1, P, 64, dtype=BF, device="cuda")
    for keys, flagged in ((MOST, 0), (MOST + 1, 16), (2 ** 31 - 1 - 256, 16)):
        err = ints([0])
        api.select_keys(*table(keys, P), w, ints([0]), keep, kept, error=err)   # a budget of 0: no key is looked at
        assert int(err) == flagged and int(kept) == 0 and keep.flatten().tolist() == [-1] * 3
        api.compact_paged_kv(*table(keys, P), ints([[[0, 1, 2]]]), ints([3]), kv, error=err)
        assert int(err) == flagged and not kv.any()


@pytest.mark.parametrize("share", [False, True])
def test_a_list_of_the_longest_kind(share):
    """max_keep 2^31 - 1: every place behind the kept keys is -1, and nothing behind the list is written."""
    n = 2 ** 31 - 1
    room = torch.zeros(n + 8192, dtype=torch.int32, device="cuda")
    keep, kept, err = room[:n].view(1, 1, n), ints([0]), ints([0])
    keys = 70000 if share else 900   # shared by a cluster's CTAs, or not
    api.select_keys(*table(keys, 16), torch.rand(1, 1, 16, device="cuda"), ints([5]), keep, kept, window=2, error=err)
    assert int(err) == 0 and int(kept) == 5
    assert keep[0, 0, 3:5].tolist() == [keys - 2, keys - 1] and int(keep[0, 0, :3].min()) >= 0
    for at in range(5, n, 2 ** 28):
        assert bool((room[at:min(at + 2 ** 28, n)] == -1).all())
    assert not room[n:].any()
