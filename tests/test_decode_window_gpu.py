"""Single tokens over the keys of a sliding window and the sinks, against float64
(bounds derived in serving_ref.py)."""

import numpy as np
import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build
from serving_ref import Cache, attend, bounds, f64

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LENS = [0, 1, 2, 63, 64, 65, 200, 511, 700, 1024]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(autouse=True)
def _status_clear():
    api.device_status()
    yield
    assert api.device_status() == _abi.JVP_OK


def queries(c, H, dt, seed=5):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(len(c.lens), H, c.D, generator=g).to(DT[dt])


def call(q, c, window, sinks, **kw):
    d = c.cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    return api.attention_decode(q.cuda(), d["k_cache"], d["v_cache"], d["block_table"], lens,
                                k_scale=d["k_scale"], v_scale=d["v_scale"], return_lse=True,
                                window=window, sinks=sinks, **kw)


def check(q, c, window, sinks, o, lse):
    B, H, D = q.shape
    tc = api.last_path() == 1
    u = torch.finfo(q.dtype).eps / 2
    w = (2.0 ** -11 if c.e4m3 else u) if tc else 0.0
    G = H // c.Hkv
    o, lse = f64(o), f64(lse)
    for b, n in enumerate(c.lens):
        j = np.arange(n)
        keep = ((j >= n - window) | (j < sinks))[None].repeat(G, 0)
        k, v = c.rows(b)
        for hk in range(c.Hkv):
            h = slice(hk * G, (hk + 1) * G)
            ref = attend(f64(q[b, h]), k[hk], v[hk], keep, D ** -0.5)
            b_o, b_lse = bounds(*ref, n, D, u, w, tc)
            assert (np.abs(o[b, h] - ref[0]) <= b_o).all(), (b, hk)
            ok = np.abs(lse[b, h] - ref[1]) <= b_lse if n else np.isneginf(lse[b, h])
            assert np.all(ok), (b, hk)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 3), (64, 0), (64, 64), (100, 130),
                                          (128, 1), (300, 4), (1000, 0), (1024, 5), (5000, 0),
                                          (2 ** 40, 2 ** 40)])
@pytest.mark.parametrize("dt,H,Hkv,D,page,e4m3", [
    ("bf16", 8, 2, 128, 16, False), ("f16", 4, 4, 64, 32, False), ("bf16", 16, 1, 128, 64, True),
    ("f16", 3, 1, 96, 24, False), ("f32", 4, 2, 64, 16, False), ("bf16", 2, 1, 60, 7, False)])
def test_windows_and_sinks(dt, H, Hkv, D, page, e4m3, window, sinks):
    c = Cache(LENS, Hkv, D, page, DT[dt], e4m3, seed=window % 97)
    q = queries(c, H, dt)
    o, lse = call(q, c, window, sinks)
    check(q, c, window, sinks, o, lse)


@pytest.mark.parametrize("dt,e4m3", [("bf16", False), ("bf16", True), ("f32", False)])
def test_hidden_keys_are_not_read(dt, e4m3):
    """Infinities and NaN in hidden positions have no say, and their pages need not exist."""
    window, sinks, page = 150, 5, 16
    c = Cache(LENS, 2, 64, page, DT[dt], e4m3, seed=2)
    q = queries(c, 4, dt)
    want = call(q, c, window, sinks)
    bad = torch.tensor([float("nan"), float("inf")]).repeat(32)
    for b, n in enumerate(c.lens):
        for j in range(sinks, n - window):
            pg, r = int(c.table[b, j // page]), j % page
            c.k[pg, :, r] = bad.to(c.k.dtype)
            c.v[pg, :, r] = bad.flip(0).to(c.v.dtype)
        for e in range(-(-sinks // page), max(0, n - window) // page):
            c.table[b, e] = -7 - e
    got = call(q, c, window, sinks)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_window_as_wide_as_the_sequence_changes_nothing(dt):
    c = Cache(LENS, 2, 128, 16, DT[dt], False, seed=4)
    q = queries(c, 8, dt)
    for a, b in zip(call(q, c, 1024, 0), call(q, c, None, 0)):
        assert torch.equal(a, b)
    for a, b in zip(call(q, c, None, 3), call(q, c, None, 0)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt,e4m3", [("f16", False), ("bf16", True)])
def test_long_sequences_are_split(dt, e4m3):
    c = Cache([30000, 77, 12345], 2, 64, 64, DT[dt], e4m3, seed=6)
    q = queries(c, 4, dt)
    o, lse = call(q, c, 9000, 700)
    check(q, c, 9000, 700, o, lse)
    for a, b in zip(call(q, c, 9000, 700), (o, lse)):
        assert torch.equal(a, b)


def test_captured_graph_follows_lengths():
    c = Cache([900, 300, 555], 2, 128, 16, torch.bfloat16, False, seed=8)
    q = queries(c, 8, "bf16").cuda()
    d = c.cuda()
    lens = torch.tensor([100, 300, 20], dtype=torch.int32).cuda()
    args = (q, d["k_cache"], d["v_cache"], d["block_table"], lens)
    api.attention_decode(*args, window=90, sinks=2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = api.attention_decode(*args, window=90, sinks=2)
    lens.copy_(torch.tensor([900, 0, 555], dtype=torch.int32))
    graph.replay()
    assert torch.equal(o, api.attention_decode(*args, window=90, sinks=2))


def test_refusals():
    c = Cache([9], 2, 64, 16, torch.bfloat16, False, seed=1)
    q = queries(c, 2, "bf16")
    for window, sinks in ((0, 0), (-1, 0), (4, -1), (None, -1)):
        with pytest.raises(ValueError):
            call(q, c, window, sinks)
    with pytest.raises(TypeError):
        call(q, c, 2.5, 0)


@pytest.mark.parametrize("window,sinks", [(5, 5000), (1, 700), (64, 65), (2 ** 40, 3)])
@pytest.mark.parametrize("dt,H,Hkv,D,page,e4m3", [
    ("bf16", 8, 2, 128, 16, False), ("f16", 4, 4, 64, 20, False), ("bf16", 16, 1, 128, 64, True),
    ("f32", 4, 2, 64, 16, False)])
def test_sinks_that_reach_into_the_window(dt, H, Hkv, D, page, e4m3, window, sinks):
    c = Cache(LENS, Hkv, D, page, DT[dt], e4m3, seed=3)
    q = queries(c, H, dt)
    o, lse = call(q, c, window, sinks)
    check(q, c, window, sinks, o, lse)
