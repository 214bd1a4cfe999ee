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


def unit_scale():
    """The scale whose logits are exact in log2 units: scale * log2(e) rounds to 1."""
    log2e = np.float32(1.4426950408889634)
    near = np.float32(1.0) / log2e
    for s in (near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(1))):
        if np.float32(s * log2e) == 1:
            return float(s)
    raise AssertionError("no such scale")


def steps(power):
    """Differences, in log2 units, that fp32 holds beside 2^power (and e4m3 beside
    the rest of a row)."""
    u = 2.0 ** (power - 23)
    return sorted({max(1, int(np.ceil(x / u))) * u for x in (4.0, 4.5, 5.0, 8.0, 16.0)})


def far_logits(n, power, step, at, D, dt):
    """q, k, v: all logits are 2^power (log2 units), that of key `at` larger by step."""
    q, k, v = torch.zeros(D), torch.zeros(n, D), torch.zeros(n, D)
    q[0], q[1] = 2.0 ** 15, 1.0
    k[:, 0], k[at, 1] = 2.0 ** (power - 15), step
    v[:, 0], v[at, 0], v[at, 1] = 1.0, 0.0, 1.0
    return [x.to(DT[dt]) for x in (q, k, v)]


def far_bounds(q, k, v, u, w):
    # (the logits are exact, products and sums too: no error of theirs)
    n, D = k.shape
    o, lse, mag, big = attend(f64(q)[None], f64(k), f64(v), np.ones((1, n), bool), np.log(2.0))
    return (o[0], lse[0]), [b[0] for b in bounds(o, lse, mag, 0 * big, n, D, u, w, True)]


@pytest.mark.parametrize("power", [12, 18, 20, 21, 22, 23, 24, 25, 26, 27])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_packed_prompts_with_large_logits(dt, D, power):
    """Where fp32 has few or no bits behind the point of a logit, weights beside a
    maximum that has not moved yet stay in range."""
    n, at, u = 300, 200, torch.finfo(DT[dt]).eps / 2
    for step in steps(power):
        q, k, v = far_logits(n, power, step, at, D, dt)
        for lens in ([n], [n] * 4 + [5 * n]):
            x = [t.expand(n, D) if t.dim() == 1 else t for t in (q, k, v)]
            x = [torch.cat([t] * (sum(lens) // n))[:, None].contiguous().cuda() for t in x]
            cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
            o, lse = api.attention_packed(*x, cu, scale=unit_scale(), return_lse=True)
            assert api.last_path() == 1
            want, tol = far_bounds(q, k, v, u, u)
            assert (np.abs(f64(o[:n, 0]) - want[0]) <= tol[0]).all(), (step, lens)
            assert (np.abs(f64(lse[0, :n]) - want[1]) <= tol[1]).all(), (step, lens)


@pytest.mark.parametrize("power", [12, 18, 20, 21, 22, 23, 24, 25, 26, 27])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [2, 12])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_single_tokens_with_large_logits(dt, H, D, power):
    """(Few keys, so that a CTA has a whole sequence: log-sum-exps of parts, by which
    they are joined, would be rounded to the steps of fp32 here.)"""
    n, at, page, B, u = 250, 201, 16, 3, torch.finfo(DT[dt]).eps / 2
    most = -(-n // page)
    for step in steps(power):
        q, k, v = far_logits(n, power, step, at, D, dt)
        kc, vc = (torch.zeros(most, 1, page, D, device="cuda", dtype=DT[dt]) for _ in range(2))
        table = torch.arange(most, dtype=torch.int32, device="cuda")
        api.cache_write(k[:, None].cuda(), v[:, None].cuda(), kc, vc, table[None],
                        cu_seqlens=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        o, lse = api.attention_decode(q.expand(B, H, D).contiguous().cuda(), kc, vc,
                                      table.expand(B, most).contiguous(),
                                      torch.full((B,), n, dtype=torch.int32, device="cuda"),
                                      scale=unit_scale(), return_lse=True)
        assert api.last_path() == 1
        want, tol = far_bounds(q, k, v, u, u)
        assert (np.abs(f64(o) - want[0]) <= tol[0]).all(), step
        assert (np.abs(f64(lse) - want[1]) <= tol[1]).all(), step


@pytest.mark.parametrize("power", [12, 20, 23, 24, 25, 26, 27])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 250])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_value_scales_beside_large_logits(dt, n, D, power):
    """An e4m3 cache whose rows of values have scales of their own."""
    at, page, B, H, u = n * 4 // 5, 16, 3, 2, torch.finfo(DT[dt]).eps / 2
    most = -(-n // page)
    for step in steps(power):
        q, k, v = far_logits(n, power, step, at, D, dt)
        v *= torch.exp2(torch.arange(n) * 7 % 9 - 4.0)[:, None]
        kc, vc = (torch.zeros(most, 1, page, D, device="cuda").to(torch.float8_e4m3fn)
                  for _ in range(2))
        ks, vs = (torch.zeros(kc.shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2))
        table = torch.arange(most, dtype=torch.int32, device="cuda")
        api.cache_write(k[:, None].cuda(), v[:, None].cuda(), kc, vc, table[None], k_scale=ks, v_scale=vs,
                        cu_seqlens=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        o, lse = api.attention_decode(q.expand(B, H, D).contiguous().cuda(), kc, vc,
                                      table.expand(B, most).contiguous(),
                                      torch.full((B,), n, dtype=torch.int32, device="cuda"),
                                      k_scale=ks, v_scale=vs, scale=unit_scale(), return_lse=True)
        assert api.last_path() == 1
        want, tol = far_bounds(q, k, v, u, 2.0 ** -11)
        assert (np.abs(f64(o) - want[0]) <= tol[0]).all(), step
        assert (np.abs(f64(lse) - want[1]) <= tol[1]).all(), step
