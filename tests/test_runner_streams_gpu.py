"""Calls on a stream of their own, with a plan made for the one call, beside work of the caller's current stream."""
import pytest
import torch

from paged_kv_cache_bsr_gb300 import api, runner, workloads as W
from kv8_util import batch, quantised, to_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("raw", [False, True])
def test_one_call_plans_on_another_stream(raw):
    """The stream is busy when the calls are made; the caller then allocates, writes and frees on the current
    one, while the calls run. Twice, so that the second round's memory is the first's."""
    b, r = batch([1] * 6, [900, 3, 4000, 77, 1, 300], seed=1), batch([70, 3, 200], [70, 500, 333], causal=True, seed=2)
    jobs = []
    for x in (b, r):
        cache, _ = quantised(x, 1, poison=False)
        jobs.append((x, runner.DeviceBatch.from_host(x), to_cuda(cache)))
    k, v = (t.cuda() for t in W.new_kv_rows(r))
    rope = api.make_rope_axes(1e4, 128, [64])
    (_, db, cb), (_, dr, cr) = jobs

    def calls(s):
        scratch = runner.Kv8Cache(cr.codes.view(torch.uint8).clone().view(torch.float8_e4m3fn), cr.scales.clone())
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        st = s.cuda_stream if raw and s is not None else s
        return (*runner.decode_kv8(db, cb, stream=st), *runner.prefill_kv8(dr, cr, stream=st), *runner.decode(db, stream=st),
                *runner.prefill(dr, stream=st), runner.append_kv8(dr, scratch, k, v, rope, stream=st)), scratch

    want, _ = calls(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    m = torch.randn(8192, 8192, device="cuda").bfloat16()
    for _ in range(2):
        with torch.cuda.stream(s):
            y = m
            for _ in range(8):
                y = y @ m
        got, keep = calls(s)
        for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24):
            for _ in range(4):
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().wait_stream(s)
        for x, w in zip(got, want):
            assert torch.equal(x, w)
        del got
    torch.cuda.synchronize()


def test_the_default_streams_raw_handle():
    b = batch([1] * 2, [90, 3], seed=3)
    cache, _ = quantised(b, 1, poison=False)
    db, c = runner.DeviceBatch.from_host(b, kv_data=torch.empty(0)), to_cuda(cache)
    want, got = runner.decode_kv8(db, c), runner.decode_kv8(db, c, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
