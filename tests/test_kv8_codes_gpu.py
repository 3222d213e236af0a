"""Codes that the append into the 8-bit cache writes, against the rotation in double precision, by the million."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_bsr_gb300 import api, runner

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_bsr_gb300 import build
    build.build()
    api.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("small", [2.0 ** -14, 2.0 ** -16, 1.0])
def test_append_codes_are_the_nearest_at_every_size(small):
    """Rows whose first pair holds the largest magnitude, the others `small` times a normal number (2^-14 puts
    them among e4m3's subnormals, where its steps are even): every turned element of at least an eighth of its
    pair's length gets the code of the exact rotation, over 60 million elements."""
    n, hkv, P, D = 30000, 8, 128, 128
    pages = (n + P - 1) // P
    g = torch.Generator("cuda").manual_seed(int(-np.log2(small)))
    cache = runner.Kv8Cache.zeros(pages, hkv, P, D)
    params = api.make_params(hkv, hkv, D, P, BF, 1.0)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ix = torch.arange(pages, dtype=torch.int32, device="cuda")
    theta = 1e4
    rope = api.make_rope_axes(theta, D, [D // 2])
    values = torch.from_numpy(oracle.e4m3_values()).cuda()
    freq = theta ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device="cuda") / D)
    off, seen = 0, 0
    for _ in range(2):
        x = torch.randn(n, hkv, D, generator=g, device="cuda") * small
        x[..., 0], x[..., D // 2] = 1.0, 0.0
        x = x.clamp(-1.0, 1.0).to(BF)
        pos = torch.randint(0, 4096, (1, n), generator=g, dtype=torch.int32, device="cuda")
        api.append_paged_kv8(params, rope, i32(0, n), i32(0, pages), ix, i32(n - (pages - 1) * P), pos, x, x, cache.codes,
                             cache.scales)
        got = values[cache.codes.view(torch.uint8)[:, 0].permute(0, 2, 1, 3).reshape(-1, hkv, D)[:n].long()]
        xd = x.double() * 128.0                                  # the largest is 1: s = 120
        assert bool((cache.scales[:, 0].permute(0, 2, 1).reshape(-1, hkv)[:n] == 120).all())
        ang = pos[0].double().unsqueeze(1) * freq
        c, s = torch.cos(ang).unsqueeze(1), torch.sin(ang).unsqueeze(1)
        u, v = xd[..., :D // 2], xd[..., D // 2:]
        r = torch.hypot(u, v)
        for half, y in ((0, u * c - v * s), (1, v * c + u * s)):
            step = torch.exp2(torch.frexp(y)[1].double().sub(1).clamp(min=-6) - 3)
            q = y / step
            # an exact element this near to a border (an angle of the reference is good to 2^-40) has two right codes
            clear = ((q - torch.floor(q) - 0.5).abs() * step > r * 2.0 ** -38) & (y.abs() >= r / 8)
            want = torch.round(q) * step
            code = got[..., half * (D // 2):(half + 1) * (D // 2)]
            off += int(((code != want) & clear).sum())
            seen += int(clear.sum())
    assert seen > 5e7 and off == 0, f"{off} of {seen} codes are not the nearest"
