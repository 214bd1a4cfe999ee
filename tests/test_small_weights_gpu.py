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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [250, 500, 3000])
@pytest.mark.parametrize("H", [4, 24])  # one or two groups of 8 query heads
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("dt,e4m3", [("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
def test_single_tokens(dt, e4m3, where, H, n, D):
    """Many sequences, so that few parts of a sequence have the far key to themselves."""
    B, Hkv, page = 300, 2, 16
    far = {"first": 0, "middle": n // 2, "last": n - 1}[where]
    q, k, v = rows(n, far, D, dt)
    u = torch.finfo(DT[dt]).eps / 2
    most = -(-n // page)
    cache = torch.float8_e4m3fn if e4m3 else DT[dt]
    kc, vc = (torch.zeros(most, Hkv, page, D, device="cuda").to(cache) for _ in range(2))
    sc = [torch.zeros(kc.shape[:3], dtype=torch.uint8, device="cuda") if e4m3 else None
          for _ in range(2)]
    table = torch.arange(most, dtype=torch.int32, device="cuda")
    api.cache_write(*(x[:, None].expand(n, Hkv, D).contiguous().cuda() for x in (k, v)), kc, vc,
                    table[None], cu_seqlens=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                    k_scale=sc[0], v_scale=sc[1])
    tables = table.expand(B, most).contiguous()  # (sequences may share pages that are only read)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    qs = q[0].expand(B, H, D).contiguous().cuda()
    for nats in NATS:
        o, lse = api.attention_decode(qs, kc, vc, tables, lens, k_scale=sc[0], v_scale=sc[1],
                                      scale=nats, return_lse=True)
        assert api.last_path() == 1
        ref = attend(f64(q[:1]), f64(k), f64(v), np.ones((1, n), bool), float(np.float32(nats)))
        b_o, b_lse = bounds(*ref, n, D, u, 2.0 ** -11 if e4m3 else u, True)
        e = np.abs(f64(o) - ref[0][0]).max((0, 1))
        assert (e <= b_o[0]).all(), (nats, (e / b_o[0]).max())
        assert (np.abs(f64(lse) - ref[1][0]) <= b_lse[0]).all(), nats
