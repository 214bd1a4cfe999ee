"""Caches and batches whose indices need more than 32 bits, or nearly as many."""

import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(autouse=True)
def _status_clear():
    api.device_status()
    yield
    assert api.device_status() == _abi.JVP_OK


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("page,Hkv", [(1 << 30, 3), ((1 << 30) - 1, 2)])
def test_scales_of_a_page_past_31_bits(page, Hkv):
    """One page of 2^30 rows and three heads: the third head's scales begin at byte
    2^31 (and a page that stays below).  Only one row of it is used; the others may
    overlap in memory."""
    D, at = 16, page - 5
    x = [torch.randn(1, Hkv, D, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() * 8.0 ** i
         for i in range(2)]
    table = i32([[0]])
    caches = [torch.empty(8 * page + 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
              .as_strided((1, Hkv, page, D), (8 * page, 16, 8, 1)) for _ in range(2)]
    scales = [torch.empty(1, Hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for s in scales:
        s[:, :, at] = 1  # (not the scale of any of these rows)
    kw = dict(k_scale=scales[0], v_scale=scales[1])
    api.cache_write(*x, *caches, table, i32([at]), **kw)
    got = api.cache_read(*caches, table, i32([at]), **kw)
    small = [torch.zeros(1, Hkv, 1, D, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    ss = [torch.zeros(1, Hkv, 1, dtype=torch.uint8, device="cuda") for _ in range(2)]
    api.cache_write(*x, *small, table, k_scale=ss[0], v_scale=ss[1])
    want = api.cache_read(*small, table, k_scale=ss[0], v_scale=ss[1])
    for i in range(2):
        assert torch.equal(scales[i][:, :, at], ss[i][:, :, 0])
        assert torch.equal(got[i], want[i])


def test_more_than_2_to_the_30_sequences():
    """Nearly all of them empty."""
    B, page, D = (1 << 30) + 40, 4, 8
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[B - 2:] = i32([1, 1, 5])  # sequence B - 3 has row 0, sequence B - 1 the others
    table = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    table[B - 3], table[B - 1] = 2, 0
    x = torch.randn(5, 1, D, device="cuda").bfloat16()
    kc, vc = (torch.zeros(3, 1, page, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    api.cache_write(x, -x, kc, vc, table, None, cu)
    assert torch.equal(kc[0], x[1:].transpose(0, 1)) and torch.equal(vc[0], -x[1:].transpose(0, 1))
    assert torch.equal(kc[2, 0, 0], x[0, 0]) and kc[2, 0, 1:].eq(0).all() and kc[1].eq(0).all()
    k, v = api.cache_read(kc, vc, table, None, cu, num_rows=5)
    assert torch.equal(k, x) and torch.equal(v, -x)
