"""Sequences whose offsets are good one by one but overlap."""

import pytest
import torch
from forward_mode_flash_gb300 import _abi, api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("dt,H,D,T,B", [
    (torch.float32, 32, 1, (1 << 22) + 1024, 2048),  # a sum of tiles past 2^32
    (torch.float32, 1, 1, 5000, 2048), (torch.bfloat16, 128, 8, 3000, 5000),
    (torch.float32, 2, 4, 40, 3), (torch.bfloat16, 4, 64, 700, 5)])
def test_every_other_pair_is_the_whole_batch(dt, H, D, T, B):
    """0, T, 0, T, ...: reported, and not worked through many times over."""
    q = torch.zeros(T, H, D, dtype=dt, device="cuda")
    k = torch.zeros(1, 1, 16, D, dtype=dt, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 16, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    api.device_status()
    api.attention_chunk(q, k, k, table, lens, cu, out=out)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    assert (out == (3.0 if B > 5 else 0.0)).all()  # (a few: the good pairs' rows)
    # and what comes next is as ever
    cu = torch.tensor([0, 2] + [2] * (B - 1), dtype=torch.int32, device="cuda")
    got = api.attention_chunk(q[:2], k + 1, k + 1, table, lens, cu)
    assert (got == 1.0).all() and api.device_status() == _abi.JVP_OK
