"""The tensors that the runner makes for a call on a given stream belong to that stream: memory of another
stream's pool could still be in use by that stream's earlier work, and a plan freed on return be reused by its next."""
import contextlib
import dataclasses

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api, runner, workloads as W
from kv8_util import batch

BF = torch.bfloat16


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Recorder:
    """Stands in for the streams, the plan and the library: notes on which stream each allocation is made."""

    def __init__(self, monkeypatch):
        self.default, self.now, self.made, self.ran, self.recorded = FakeStream(0), [], [], [], []
        rec = self

        @contextlib.contextmanager
        def on(stream):
            rec.now.append(stream)
            yield
            rec.now.pop()

        class FakePlan:
            def __init__(self, kind):
                self.kind = kind
                rec.made.append(rec.current().cuda_stream)

            def plan(self, *a, stream=None, **k):
                rec.ran.append(stream)

            def run(self, *a, stream=None, **k):
                rec.ran.append(stream)

        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: rec.current())
        monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
        monkeypatch.setattr(runner, "make_plan", lambda b, kind, **k: FakePlan(kind))
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: rec.recorded.append(s.cuda_stream))
        for name in ("empty", "empty_like"):
            monkeypatch.setattr(torch, name, self.wrap(getattr(torch, name)))
        for name in ("append_paged_kv", "append_paged_kv_axes", "append_paged_kv8", "merge_state", "merge_states"):
            monkeypatch.setattr(api, name, lambda *a, stream=None, **k: rec.ran.append(stream))

    def current(self):
        return self.now[-1] if self.now else self.default

    def wrap(self, fn):
        def alloc(*a, **k):
            self.made.append(self.current().cuda_stream)
            return fn(*a, **k)
        return alloc


def calls():
    one, rows = batch([1, 1], [20, 3], seed=1), batch([4, 3], [20, 3], seed=2)
    dev = lambda b: runner.DeviceBatch(b, b.q, b.kv_data, b.qo_indptr, b.kv_indptr, b.kv_indices, b.kv_last_page_len)
    cache = runner.Kv8Cache(torch.zeros(rows.num_pages, 2, 2, 16, 128, dtype=torch.uint8),
                            torch.zeros(rows.num_pages, 2, 2, 16, dtype=torch.uint8))
    k, v = W.new_kv_rows(rows)
    a, r = dev(one), dev(rows)
    return {"decode": lambda s: runner.decode(a, stream=s), "prefill": lambda s: runner.prefill(r, stream=s),
            "mixed": lambda s: runner.mixed(r, stream=s), "decode_kv8": lambda s: runner.decode_kv8(a, cache, stream=s),
            "prefill_kv8": lambda s: runner.prefill_kv8(r, cache, stream=s),
            "cascade": lambda s: runner.cascade(a, a, stream=s), "cascade_kv8": lambda s: runner.cascade_kv8(a, a, cache, stream=s),
            "levels_mixed": lambda s: runner.levels_mixed(a, 2, stream=s),
            "multi_level_cascade": lambda s: runner.multi_level_cascade([a, a], stream=s),
            "append_kv": lambda s: runner.append_kv(r, k, v, stream=s),
            "append_kv_axes": lambda s: runner.append_kv_axes(r, k, v, None, stream=s),
            "append_kv8": lambda s: runner.append_kv8(r, cache, k, v, stream=s)}


@pytest.mark.parametrize("name", sorted(calls()))
@pytest.mark.parametrize("raw", [False, True])
def test_allocations_are_made_on_the_calls_stream(monkeypatch, name, raw):
    fn = calls()[name]
    rec = Recorder(monkeypatch)
    s = 77 if raw else FakeStream(77)
    fn(s)
    assert rec.made and set(rec.made) == {77}
    assert rec.ran and all(x is s for x in rec.ran)
    assert rec.recorded and set(rec.recorded) == {0}    # what is returned outlives its use on the caller's stream too


@pytest.mark.parametrize("name", sorted(calls()))
def test_calls_without_a_stream_use_the_current_one(monkeypatch, name):
    fn = calls()[name]
    rec = Recorder(monkeypatch)
    fn(None)
    assert rec.made and set(rec.made) == {0} and not rec.recorded
