"""What the binding takes as an 8-bit cache."""
import pytest
import torch

from paged_kv_cache_bsr_gb300 import api

CODES = (4, 2, 2, 16, 128)
OTHERS = [torch.int8, torch.bool, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.float16]


def params():
    return api.make_params(8, 2, 128, 16, torch.bfloat16, 0.1)


@pytest.mark.parametrize("dtype", OTHERS)
def test_pools_of_other_types_are_refused(dtype):
    """Codes of another 8-bit type would be read as e4m3."""
    rows = lambda n, h: torch.zeros(n, h, 128, dtype=torch.bfloat16)
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    kv8 = torch.zeros(CODES).to(dtype)
    with pytest.raises(ValueError, match="float8_e4m3fn or uint8"):
        api.append_paged_kv8(params(), None, i(3), i(3), i(4), i(2), None, rows(5, 2), rows(5, 2), kv8,
                             torch.zeros(CODES[:-1], dtype=torch.uint8))
    with pytest.raises(ValueError, match="float8_e4m3fn or uint8"):
        api._kv8_tensors(params(), kv8, torch.zeros(CODES[:-1], dtype=torch.uint8))


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn])
def test_pools_of_e4m3_codes_are_taken(dtype):
    codes = torch.zeros(CODES, dtype=torch.uint8).view(dtype)
    api._kv8_tensors(params(), codes, torch.zeros(CODES[:-1], dtype=torch.uint8))
    with pytest.raises(ValueError):
        api._kv8_tensors(params(), codes, torch.zeros(CODES[:-1], dtype=torch.int8))
