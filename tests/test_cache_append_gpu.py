"""Keys and values into a paged cache with the norms and rotation on the way."""

import numpy as np
import pytest
import torch

import rope_ref
from forward_mode_flash_gb300 import _abi, api, build
from serving_ref import Cache

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(autouse=True)
def _status_clear():
    api.device_status()
    yield
    assert api.device_status() == _abi.JVP_OK


def case(new, past, H, Hkv, D, dt, cache="", page=16, rot=None, norm=True, seed=0, behind=0):
    """Inputs of a call; the cache's rows are made new."""
    g = torch.Generator().manual_seed(seed)
    T = sum(new) + behind
    total = [a + b for a, b in zip(new, past)]
    c = Cache(total, Hkv, D, page, DT[dt], cache == "e4m3", seed)
    x = {n: torch.randn(T, h, D, generator=g).to(DT[dt]).cuda()
         for n, h in (("q", H), ("k", Hkv), ("v", Hkv))}
    rot = D if rot is None else rot
    w = [1 + 0.3 * torch.randn(D, generator=g).cuda() for _ in range(2)] if norm else [None, None]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    start = torch.tensor(past, dtype=torch.int32).cuda()
    table = api.rope_table(max(total + [1]), rot, device="cuda") if rot else None
    return c, x, w, cu, start, table


def append(c, x, w, cu, start, table, interleaved=False, **kw):
    d = c.cuda()
    q = api.cache_append(x["q"], x["k"], x["v"], d["k_cache"], d["v_cache"], d["block_table"], table,
                         start, cu, *w, EPS, interleaved, d["k_scale"], d["v_scale"], **kw)
    return q, d


def check(c, x, w, new, past, table, q, d, interleaved):
    """Against the dense kernel (which has its own tests) and a write of its result."""
    T = sum(new)
    pos = torch.tensor([p + i for n, p in zip(new, past) for i in range(n)], dtype=torch.int32)
    one = lambda t: t[:T].transpose(0, 1)[None]  # noqa: E731  [1, H, T, D]
    rq, rk = api.norm_rope(one(x["q"]), one(x["k"]), table, pos.cuda(), *w, EPS, interleaved)
    assert torch.equal(q[:T], rq[0].transpose(0, 1))
    e = c.cuda()
    k = torch.zeros_like(x["k"])
    k[:T] = rk[0].transpose(0, 1)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    api.cache_write(k, x["v"], e["k_cache"], e["v_cache"], e["block_table"],
                    torch.tensor(past, dtype=torch.int32).cuda(), cu, e["k_scale"], e["v_scale"])
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if d[n] is not None:
            assert torch.equal(d[n].view(torch.uint8), e[n].view(torch.uint8)), n


@pytest.mark.parametrize("cache", ["", "e4m3"])
@pytest.mark.parametrize("norm,interleaved", [(True, False), (False, False), (True, True), (False, True)])
@pytest.mark.parametrize("dt,H,Hkv,D,rot", [
    ("bf16", 8, 2, 128, 128), ("f16", 4, 4, 64, 32), ("f32", 6, 2, 128, 128), ("f32", 2, 1, 64, 64),
    ("bf16", 5, 1, 80, 80), ("f16", 3, 3, 40, 40), ("bf16", 2, 2, 96, 64), ("f32", 3, 1, 33, 6),
    ("bf16", 7, 1, 2, 2), ("f16", 0, 2, 64, 64)])
def test_rows_as_the_dense_kernel_and_a_write_leave_them(dt, H, Hkv, D, rot, norm, interleaved, cache):
    new, past = [1, 0, 17, 40, 3], [5, 9, 0, 100, 31]
    a = case(new, past, H, Hkv, D, dt, cache, rot=rot, norm=norm, seed=D)
    q, d = append(*a, interleaved=interleaved)
    check(a[0], a[1], a[2], new, past, a[5], q, d, interleaved)


@pytest.mark.parametrize("page", [1, 8, 24, 64])
@pytest.mark.parametrize("dt,cache", [("bf16", ""), ("bf16", "e4m3"), ("f32", "")])
def test_pages_and_a_padded_batch(dt, cache, page):
    new, past = [30, 1, 65], [0, 77, 10]
    a = case(new, past, 4, 2, 64, dt, cache, page=page, behind=7)
    out = torch.full_like(a[1]["q"], 3.0)
    q, d = append(*a, out=out)
    assert q.data_ptr() == out.data_ptr()
    check(a[0], a[1], a[2], new, past, a[5], q, d, False)
    assert (out[-7:] == 3.0).all()


def test_norms_alone_and_single_tokens():
    past = [3, 200, 0, 15]
    c, x, w, _, start, _ = case([1] * 4, past, 8, 2, 128, "bf16")
    q, d = append(c, x, w, None, start, None)
    check(c, x, w, [1] * 4, past, None, q, d, False)


def test_a_row_against_float64():
    """(The comparison above is with the dense kernel; this one with the definition.)"""
    new, past = [9, 4], [2, 300]
    c, x, w, cu, start, table = case(new, past, 4, 2, 128, "bf16", seed=3)
    q, d = append(c, x, w, cu, start, table)
    pos = torch.tensor([2 + i for i in range(9)] + [300 + i for i in range(4)])
    at = table.cpu()[pos][:, None]
    zero = torch.zeros(13, 1, 128)
    rope_ref.check_side({"y": q.cpu()}, x["q"].cpu(), None, zero, None, w[0].cpu(), at, EPS, False)
    rk, rv = api.cache_read(d["k_cache"], d["v_cache"], d["block_table"], start, cu, num_rows=13)
    rope_ref.check_side({"y": rk.cpu()}, x["k"].cpu(), None, zero, None, w[1].cpu(), at, EPS, False)
    assert torch.equal(rv, x["v"])


def test_places_out_of_range_are_skipped_and_reported():
    new, past = [3, 2, 2], [4, 0, 1]
    c, x, w, cu, start, table = case(new, past, 2, 1, 64, "bf16")
    good = append(c, x, w, cu, start, table, out=torch.zeros_like(x["q"]))
    # a position behind the table of angles, and a page that does not exist
    c.table[1, 0] = c.pages
    d = c.cuda()
    out = torch.zeros_like(x["q"])
    api.cache_append(x["q"], x["k"], x["v"], d["k_cache"], d["v_cache"], d["block_table"],
                     table[:6], start, cu, *w, EPS, out=out)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    keep = torch.tensor([0, 1, 5, 6]).cuda()  # positions 4, 5 of the first, 1, 2 of the third
    assert torch.equal(out[keep], good[0][keep])
    assert (out[[2, 3, 4]] == 0).all()
    # offsets that decrease, and a start before the first position
    bad = torch.tensor([0, 3, 2, 7], dtype=torch.int32).cuda()
    out.zero_()
    api.cache_append(x["q"], x["k"], x["v"], d["k_cache"], d["v_cache"], d["block_table"], table,
                     torch.tensor([-2, 0, 0], dtype=torch.int32).cuda(), bad, *w, EPS, out=out)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    assert (out[:2] == 0).all()


def test_no_rows():
    c, x, w, cu, start, table = case([0, 0], [3, 4], 2, 1, 64, "bf16")
    q, d = append(c, x, w, cu, start, table)
    assert q.shape == (0, 2, 64)
    assert torch.equal(d["k_cache"].cpu(), c.k)


def test_captured_graph_follows_positions():
    past = [3, 60, 0, 15]
    c, x, w, _, start, table = case([1] * 4, [70] * 4, 8, 2, 128, "bf16")
    start = torch.tensor(past, dtype=torch.int32).cuda()
    append(c, x, w, None, start, table)
    d = c.cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    args = (x["q"], x["k"], x["v"], d["k_cache"], d["v_cache"], d["block_table"], table, start, None,
            *w, EPS)
    with torch.cuda.graph(graph):
        q = api.cache_append(*args)
    start += 1
    graph.replay()
    want = q.clone()
    got, e = append(c, x, w, None, start, table)
    assert torch.equal(got, want) and torch.equal(e["k_cache"], d["k_cache"])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt,D,rot", [("bf16", 128, 128), ("f16", 64, 32), ("f32", 33, 6), ("bf16", 40, 20)])
def test_queries_in_place(dt, D, rot, interleaved):
    a = case([30, 1], [3, 70], 4, 2, D, dt, rot=rot, seed=6)
    want, _ = append(*a, interleaved=interleaved)
    got, _ = append(*a, interleaved=interleaved, out=a[1]["q"])
    assert got.data_ptr() == a[1]["q"].data_ptr() and torch.equal(got, want)
