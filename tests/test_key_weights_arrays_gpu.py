"""GPU tests: arrays that do not fit are always flagged by the key weights' call, whichever kernel it takes."""
import pytest
import torch

from paged_kv_cache_bsr_gb300 import api
from length_util import Paged, ints, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


def call(x, lse, before, causal):
    w, err = before.clone(), ints([0])
    p = api.make_params(x.hkv * x.group, x.hkv, x.d, x.P, x.dtype, x.d ** -0.5, 0.0, causal)
    api.add_key_weights(p, x.indptr, x.indices, x.last, x.q, lse, x.kv, w, qo_indptr=x.qo, kv_scales=x.scales, error=err)
    return w, int(err)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("qo,causal", [(None, False), ([3, 2, 4, 1], True), ([90, 60, 70, 40], True), ([90, 60, 70, 40], False)])
def test_row_pointers_that_do_not_ascend(qo, causal, kv8):
    """A row pointer set down, below 0 or past the list: flagged, and every key is as it was or as it should be."""
    x = Paged([48, 40, 64, 33], 16, 2, kv8=kv8, qo_lens=qo, group=4, seed=1)   # 3, 3, 4 and 3 pages
    lse = x.lse(x.d ** -0.5, 0.0, causal and qo is not None)
    before = torch.rand(x.pool, x.hkv, x.P, device="cuda") + 50
    good, err = call(x, lse, before, causal)
    assert err == 0
    indptr = starts([3, 3, 4, 3])
    for at, value in [(4, 3), (4, 6), (4, 0), (4, -7), (4, 14), (4, 10 ** 6), (0, -1), (0, 4), (3, 14), (2, -5), (2, 10 ** 6), (1, -2 ** 31),
                      (3, 2 ** 31 - 1)]:
        x.indptr.copy_(ints(indptr[:at] + [value] + indptr[at + 1:]))
        w, err = call(x, lse, before, causal)
        assert err == 16, (at, value)
        assert bool(((w == before) | (w == good)).all()), (at, value)
    x.indptr.copy_(ints(indptr))
    if qo is not None:
        for at, value in [(4, 10 ** 6), (4, -1), (2, -5), (2, 10 ** 6), (0, -3)]:
            was = int(x.qo[at])
            x.qo[at] = value
            w, err = call(x, lse, before, causal)
            assert err == 16 and bool(torch.isfinite(w).all()), (at, value)
            x.qo[at] = was


@pytest.mark.parametrize("batch", [200, 3000])
def test_any_one_of_many_requests(batch):
    """More requests than a warp or a block looks at."""
    lens = [(i * 7) % 33 + 1 for i in range(batch)]
    for qo in (None, [40] * batch):
        x = Paged(lens, 16, 1, qo_lens=qo, group=1, d=128, seed=2)
        lse = torch.zeros(x.q.shape[:2], device="cuda")
        before = torch.zeros(x.pool, 1, 16, device="cuda")
        for b in (0, 31, 32, 191, 192, batch // 2, batch - 1):
            if b >= batch:
                continue
            was = int(x.last[b])
            x.last[b] = 17
            assert call(x, lse, before, False)[1] == 16, b
            x.last[b] = was
        assert call(x, lse, before, False)[1] == 0
