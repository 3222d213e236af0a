"""Queries turned into memory that overlaps them: in place, or not at all."""
import ctypes

import pytest
import torch

from paged_kv_cache_bsr_gb300 import api

INVALID = -1


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    return api.load()


@pytest.mark.parametrize("kv8", [False, True])
def test_appends_refuse_queries_that_overlap_their_outputs(lib, kv8):
    """Tokens are read ahead of those that are written: 5 tokens of 8 heads of 128 16-bit elements are 10240 bytes."""
    buf = torch.zeros(65536, dtype=torch.uint8)
    base = buf.data_ptr() + (-buf.data_ptr()) % 256
    p = lambda at: ctypes.c_void_p(base + at)
    params = api.make_params(8, 2, 128, 16, torch.bfloat16, 0.1)
    fn = lib.pkv_append_paged_kv8 if kv8 else lib.pkv_append_paged_kv_axes

    def append(q_in, q_out):
        args = [ctypes.byref(params), None, 2, 5, 10, p(0), p(0), p(0), p(0), None, p(0), p(0), p(0)]
        return fn(*args, *([p(0)] if kv8 else []), p(q_in), p(q_out), None, None)

    for q_in, q_out in ((0, 16), (16, 0), (0, 10224), (10224, 0), (2048, 4096)):
        assert append(q_in, q_out) == INVALID
    if not torch.cuda.is_available():   # (a call that passes the checks is launched)
        for q_in, q_out in ((0, 10240), (20480, 10240), (4096, 4096)):
            assert append(q_in, q_out) != INVALID
