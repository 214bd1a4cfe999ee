"""Windows that a CTA reads by itself or shares, on both sides of where that changes."""

import numpy as np
import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build
from serving_ref import Cache
from test_decode_window_gpu import call, check, queries

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(autouse=True)
def _status_clear():
    api.device_status()
    yield
    assert api.device_status() == _abi.JVP_OK


# sequences times key/value heads: more than a GPU has SMs, and few
MANY = [(170, 8, 1), (42, 16, 4), (165, 16, 1), (80, 4, 2)]
FEW = [(3, 8, 1), (5, 16, 1), (2, 16, 4)]


@pytest.mark.parametrize("window,sinks", [(260, 0), (400, 3), (640, 0), (700, 70), (1020, 1), (1100, 0), (1300, 2)])
@pytest.mark.parametrize("dt,D,e4m3", [("bf16", 128, False), ("f16", 96, False), ("bf16", 64, False),
                                       ("bf16", 128, True), ("f16", 96, True), ("bf16", 64, True)])
@pytest.mark.parametrize("many", [True, False], ids=["many", "few"])
def test_windows_of_many_segments(many, dt, D, e4m3, window, sinks):
    B, H, Hkv = (MANY if many else FEW)[(window + D) % len(MANY if many else FEW)]
    lens = np.random.default_rng(window + D).integers(0, 1500, B).tolist()
    lens[0], lens[-1] = 1500, 0
    c = cache(tuple(lens), Hkv, D, dt, e4m3)
    q = queries(c, H, dt)
    o, lse = call(q, c, window, sinks)
    assert api.last_path() == 1
    check(q, c, window, sinks, o, lse)
    for a, b in zip(call(q, c, window, sinks), (o, lse)):
        assert torch.equal(a, b)


def cache(lens, Hkv, D, dt, e4m3):
    """Random pages.  e4m3: codes and scales drawn as they are."""
    c = Cache(lens, Hkv, D, 16, DT[dt], False, seed=D)
    if e4m3:
        g = torch.Generator().manual_seed(D)
        c.e4m3 = True
        c.k, c.v = (x.float().mul(100).clamp(-448, 448).to(torch.float8_e4m3fn) for x in (c.k, c.v))
        c.scales = [torch.randint(115, 122, c.k.shape[:3], generator=g).to(torch.uint8) for _ in range(2)]
    return c
