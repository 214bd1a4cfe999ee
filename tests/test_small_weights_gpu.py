"""One key far above thousands of others that share the rest of the weight.

A weight that goes to the tensor cores in fp16 must keep its relative precision
(the bounds of serving_ref.py count on it) however small it is beside the row's
largest: the weights here are 2^-26 = e^-18 of it and more, and with the factor
2^11 that the kernels give them at least 2^-15, where half a step of fp16 (2^-25)
is 2^-10 of the weight.  That is 2 w, and what the bounds allow: w for weights in
the sum and w for the row sum, which has the unrounded ones.  The far key's value
is 0 in every column but the first, so the other columns are the small weights'
alone.
"""

import numpy as np
import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build
from serving_ref import attend, bounds, f64

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
NATS = [9.3, 12.4, 15.2, 16.9, 17.3, 18.0]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(autouse=True)
def _status_clear():
    api.device_status()
    yield
    assert api.device_status() == _abi.JVP_OK


def rows(n, far, D, dt):
    """q, k, v [n, D]: every logit is 0 but those of key `far`, which are the scale."""
    q, k, v = torch.zeros(n, D), torch.zeros(n, D), torch.ones(n, D)
    q[:, 0], k[far, 0] = 1.0, 1.0
    v[:, 0] = 0.0
    v[:, 2] = 0.75
    v[far] = 0.0
    v[far, 0] = 1.0
    return [x.to(DT[dt]) for x in (q, k, v)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[2100, 3], [400, 77, 129]], ids=["two_tiles", "one_tile"])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_packed_prompts(dt, where, lens, D, causal):
    far = {"first": 0, "middle": lens[0] // 2, "last": lens[0] - 1}[where]
    parts = [rows(n, far if b == 0 else 0, D, dt) for b, n in enumerate(lens)]
    q, k, v = (torch.cat([p[i] for p in parts])[:, None] for i in range(3))
    q = q.expand(-1, 2, D).contiguous()  # two query heads on one key/value head
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    u = torch.finfo(DT[dt]).eps / 2
    n = lens[0]
    keep = np.tril(np.ones((n, n), bool)) if causal else np.ones((n, n), bool)
    for nats in NATS:
        o, lse = api.attention_packed(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), is_causal=causal,
                                      scale=nats, return_lse=True)
        assert api.last_path() == 1
        nats32 = float(np.float32(nats))
        ref = attend(f64(q[:n, 0]), f64(k[:n, 0]), f64(v[:n, 0]), keep, nats32)
        b_o, b_lse = bounds(*ref, n, D, u, u, True)
        for h in range(2):
            e = np.abs(f64(o[:n, h]) - ref[0])
            assert (e <= b_o).all(), (nats, h, (e / b_o).max())
            assert (np.abs(f64(lse[h, :n]) - ref[1]) <= b_lse).all(), (nats, h)
