"""Rows into and out of the paged cache, and single-token attention over it,
against the definitions in float64 (bounds derived in serving_ref.py)."""

import ctypes

import numpy as np
import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build
from serving_ref import Cache, attend, bounds, f64, quantise, round_e4m3

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


def cu_of(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# ------------------------------------------------------------------ write and read
CASES = [  # rows per sequence, start, Hkv, D, page, dtype, e4m3
    ([1], [0], 1, 64, 16, "bf16", False),
    ([3, 0, 17, 1], [0, 5, 9, 30], 4, 128, 16, "bf16", True),
    ([3, 0, 17, 1], [0, 5, 9, 30], 4, 128, 16, "f16", False),
    ([40, 7], [1, 0], 3, 96, 24, "f32", True),
    ([40, 7], [1, 0], 3, 96, 24, "f32", False),
    ([5, 6, 2], [0, 0, 3], 2, 40, 7, "bf16", True),     # 5 lanes of 16 bytes
    ([5, 6, 2], [0, 0, 3], 2, 20, 1, "f16", True),      # no 16-byte rows
    ([5, 6, 2], [0, 0, 3], 2, 33, 3, "bf16", False),    # odd rows
    ([5, 6, 2], [0, 0, 3], 5, 1, 3, "f32", True),
    ([130], [70], 9, 128, 64, "bf16", True),            # more heads than one pass
    ([0, 0], [0, 0], 2, 64, 16, "bf16", True),
]


@pytest.mark.parametrize("rows,start,Hkv,D,page,dt,e4m3", CASES)
def test_write_places_every_row_and_read_brings_it_back(rows, start, Hkv, D, page, dt, e4m3):
    lens = [s + r for s, r in zip(start, rows)]
    c = Cache(lens, Hkv, D, page, DT[dt], e4m3, seed=3)
    T = sum(rows)
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(T, Hkv, D, generator=g).to(DT[dt]) for _ in range(2))
    dev = c.cuda()
    before = {n: (t.clone() if t is not None else None) for n, t in dev.items()}
    cu, st = cu_of(rows), i32(start)
    api.cache_write(k.cuda(), v.cuda(), dev["k_cache"], dev["v_cache"], dev["block_table"], st, cu,
                    k_scale=dev["k_scale"], v_scale=dev["v_scale"])
    # expected caches: the old ones with the new rows put in
    for x, name, sname in ((k, "k_cache", "k_scale"), (v, "v_cache", "v_scale")):
        want = before[name].cpu().double().numpy()
        scale = before[sname].cpu().numpy().astype(np.int64) if e4m3 else None
        at = 0
        for b, n in enumerate(rows):
            for r in range(n):
                pos = start[b] + r
                pg = int(c.table[b, pos // page])
                row = x[at].double().numpy()
                if e4m3:
                    row, e = quantise(row)
                    scale[pg, :, pos % page] = e + 127
                want[pg, :, pos % page] = row
                at += 1
        np.testing.assert_array_equal(f64(dev[name].float()), want)
        if e4m3:
            np.testing.assert_array_equal(dev[sname].cpu().numpy(), scale)
    # reading the same places gives the written values
    out = api.cache_read(dev["k_cache"], dev["v_cache"], dev["block_table"], st, cu, num_rows=T,
                         k_scale=dev["k_scale"], v_scale=dev["v_scale"], dtype=DT[dt])
    for x, y in zip((k, v), out):
        want = x.double().numpy()
        if e4m3 and T:
            codes, e = quantise(want)
            want = f64(torch.from_numpy(codes * np.exp2(e)[..., None]).to(DT[dt]))
        np.testing.assert_array_equal(f64(y), want.reshape(y.shape))


def test_write_of_single_tokens_without_offsets():
    c = Cache([9, 4, 16], 2, 64, 8, torch.bfloat16, True, seed=1)
    dev = c.cuda()
    k, v = (torch.randn(3, 2, 64).to(torch.bfloat16).cuda() for _ in range(2))
    api.cache_write(k, v, dev["k_cache"], dev["v_cache"], dev["block_table"], i32([8, 3, 15]),
                    k_scale=dev["k_scale"], v_scale=dev["v_scale"])
    rk, rv = api.cache_read(dev["k_cache"], dev["v_cache"], dev["block_table"], i32([8, 3, 15]),
                            k_scale=dev["k_scale"], v_scale=dev["v_scale"])
    for x, y in ((k, rk), (v, rv)):
        codes, e = quantise(f64(x))
        np.testing.assert_array_equal(f64(y), codes * np.exp2(e)[..., None])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 20])
def test_quantisation_at_its_edges(dt, D):
    """Ties, the largest code, zeros, subnormals, NaN and infinities."""
    fi = torch.finfo(DT[dt])
    rows = [np.zeros(D), np.full(D, 448.0), np.linspace(-1, 1, D), np.full(D, fi.tiny),
            np.full(D, fi.max), np.full(D, fi.smallest_normal / 4),
            np.resize([448.0, 449.0 if dt == "f32" else 452.0, 1.0], D),   # just above 1.75 * 2^8
            np.resize([256.0, 17.0, 19.0, 21.0, 23.0, 0.0146484375, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10], D),
            np.resize([np.nan, 1.0, -3.0], D), np.resize([np.inf, 1.0, -3.0], D),
            np.resize([-np.inf, np.nan, 5.0], D), np.resize([-0.0, 2.0], D)]
    x = torch.tensor(np.array(rows)).to(DT[dt]).view(len(rows), 1, D)
    kc = torch.zeros(2, 1, 16, D, dtype=torch.float8_e4m3fn, device="cuda")
    ks = torch.zeros(2, 1, 16, dtype=torch.uint8, device="cuda")
    vc, vs = torch.zeros_like(kc), torch.zeros_like(ks)
    table, cu = i32([[1]]), cu_of([len(rows)])
    api.cache_write(x.cuda(), (-x).cuda(), kc, vc, table, None, cu, k_scale=ks, v_scale=vs)
    codes, e = quantise(f64(x))
    np.testing.assert_array_equal(ks.cpu().numpy()[1, 0, :len(rows)], (e + 127)[:, 0])
    got = f64(kc.float())[1, 0, :len(rows)]
    want = codes[:, 0]
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(np.nan_to_num(got), np.nan_to_num(want))
    np.testing.assert_array_equal(np.signbit(got[-1]), np.signbit(want[-1]))
    rk, _ = api.cache_read(kc, vc, table, None, cu, num_rows=len(rows), k_scale=ks, v_scale=vs,
                           dtype=torch.float32)
    with np.errstate(over="ignore"):
        val = (codes * np.exp2(e)[..., None]).astype(np.float32)
    np.testing.assert_array_equal(rk.cpu().numpy(), val)


def test_rounding_of_every_half_way_point():
    """All midpoints between neighbouring e4m3 values, and their float neighbours."""
    v = np.arange(127, dtype=np.uint8)
    vals = f64(torch.from_numpy(v).view(torch.float8_e4m3fn).float())
    mid = ((vals[1:] + vals[:-1]) / 2).astype(np.float32)
    x = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))])
    x = np.concatenate([x, np.zeros(-len(x) % 127, np.float32)]).reshape(-1, 127)
    x = np.concatenate([x, np.full((len(x), 1), 448.0, np.float32)], 1)  # scale 1 for each row
    t = torch.from_numpy(x).view(len(x), 1, 128).cuda()
    kc = torch.zeros(1, 1, 16, 128, dtype=torch.float8_e4m3fn, device="cuda")
    ks = torch.zeros(1, 1, 16, dtype=torch.uint8, device="cuda")
    api.cache_write(t, t, kc, kc.clone(), i32([[0]]), None, cu_of([len(x)]), k_scale=ks,
                    v_scale=ks.clone())
    assert (ks[0, 0, :len(x)] == 127).all()
    np.testing.assert_array_equal(f64(kc.float())[0, 0, :len(x)], round_e4m3(x.astype(np.float64)))


def test_strided_rows_and_caches_and_rows_outside_every_sequence():
    # q, k, v of one projection side by side; a cache with heads innermost
    # but one; rows before the first and behind the last sequence
    T, Hkv, D, page = 23, 2, 64, 8
    qkv = torch.randn(T, 3 * Hkv, D, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    base = torch.zeros(6, page, Hkv, 2 * D, device="cuda", dtype=torch.bfloat16)
    kc, vc = base[..., :D].transpose(1, 2), base[..., D:].transpose(1, 2)
    table = i32([[4, 1, -1], [0, 5, -1]])
    cu = i32([2, 12, 20])
    api.cache_write(k, v, kc, vc, table, None, cu)
    want = torch.zeros_like(base)
    for b, pages in enumerate(([4, 1], [0, 5])):
        for r in range(int(cu[b + 1] - cu[b])):
            src = int(cu[b]) + r
            want[pages[r // page], r % page, :, :D] = k[src]
            want[pages[r // page], r % page, :, D:] = v[src]
    assert torch.equal(base, want)
    out = torch.full((T, 4 * Hkv, D), 7.0, device="cuda", dtype=torch.bfloat16)
    ok, ov = out[:, Hkv:2 * Hkv], out[:, 3 * Hkv:]
    api.cache_read(kc, vc, table, None, cu, out=(ok, ov))
    keep = torch.full_like(out, 7.0)
    keep[2:20, Hkv:2 * Hkv], keep[2:20, 3 * Hkv:] = k[2:20], v[2:20]
    assert torch.equal(out, keep)


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_without_a_place_are_skipped_and_reported(e4m3):
    Hkv, D, page = 2, 64, 4
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc = torch.zeros(3, Hkv, page, D, device="cuda").to(dt)
    vc = torch.zeros(3, Hkv, page, D, device="cuda").to(dt)
    sc = [torch.zeros(3, Hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2)] if e4m3 else [None] * 2
    x = torch.ones(6, Hkv, D, device="cuda", dtype=torch.bfloat16)
    # page 3 does not exist; entry -1; position behind the table; negative position
    table = i32([[3, 0], [-1, 1], [2, 2], [2, 2], [2, 0], [2, -7]])
    api.cache_write(x, x, kc, vc, table, i32([0, 1, 8, -1, 2, 5]), None, k_scale=sc[0], v_scale=sc[1])
    assert api.device_status() == _abi.JVP_ERR_INDEX
    got = kc.float()
    assert got[2, :, 2].eq(256.0 if e4m3 else 1.0).all()  # 1 = 256 * 2^-8
    got[2, :, 2] = 0
    assert got.eq(0).all()
    out = torch.full((6, Hkv, D), 3.0, device="cuda", dtype=torch.bfloat16)
    api.cache_read(kc, vc, table, i32([0, 1, 8, -1, 2, 5]), None, k_scale=sc[0], v_scale=sc[1],
                   out=(out, out.clone()))
    assert api.device_status() == _abi.JVP_ERR_INDEX
    assert out[4].eq(1.0).all()
    out[4] = 3.0
    assert out.eq(3.0).all()


# ------------------------------------------------------------------ single tokens
def check_decode(c, q, o, lse, scale, tensor_cores, lens=None):
    lens = c.lens if lens is None else lens
    B, H, D = q.shape
    G = H // c.Hkv
    u = torch.finfo(q.dtype).eps / 2
    w = 0.0
    if tensor_cores:  # fp16 weights over e4m3, else the cache's type
        w = 2.0 ** -11 if c.e4m3 else u
    for b in range(B):
        k, v = c.rows(b, lens[b])
        for h in range(H):
            keep = np.ones((1, lens[b]), dtype=bool)
            r = attend(f64(q[b, h])[None], k[h // G], v[h // G], keep, scale)
            b_o, b_lse = bounds(*r, lens[b], D, u, w, tensor_cores)
            e_o = np.abs(f64(o[b, h]) - r[0][0])
            assert (e_o <= b_o[0]).all(), (b, h, e_o.max(), b_o[0][e_o.argmax()])
            if lens[b] == 0:
                assert np.isneginf(f64(lse[b, h]))
            else:
                assert abs(f64(lse[b, h]) - r[1][0]) <= b_lse[0], (b, h)


def decode(c, q, lens=None, **kw):
    dev = c.cuda()
    lens = i32(c.lens if lens is None else lens)
    return api.attention_decode(q.cuda(), dev["k_cache"], dev["v_cache"], dev["block_table"], lens,
                                k_scale=dev["k_scale"], v_scale=dev["v_scale"], return_lse=True, **kw)


LENS = [1, 0, 15, 16, 17, 63, 64, 65, 130, 700]


@pytest.mark.parametrize("dt,e4m3", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("H,Hkv,D,page", [(4, 4, 64, 16), (16, 4, 128, 16), (16, 1, 128, 64),
                                          (7, 1, 64, 24), (12, 2, 96, 1), (9, 1, 128, 5),
                                          (40, 2, 64, 32), (6, 2, 48, 128)])
def test_decode_on_the_tensor_cores(dt, e4m3, H, Hkv, D, page):
    c = Cache(LENS, Hkv, D, page, DT[dt], e4m3, seed=H + D)
    q = torch.randn(len(LENS), H, D, generator=torch.Generator().manual_seed(2)).to(DT[dt])
    o, lse = decode(c, q)
    assert api.last_path() == 1
    check_decode(c, q, o, lse, D ** -0.5, True)


@pytest.mark.parametrize("dt,e4m3,H,Hkv,D,page", [
    ("f32", False, 4, 4, 64, 16), ("f32", False, 16, 4, 128, 16), ("f32", True, 10, 2, 128, 7),
    ("f32", False, 3, 1, 33, 5), ("bf16", False, 6, 2, 20, 16), ("f16", True, 5, 5, 40, 3),
    ("bf16", True, 4, 2, 1, 16), ("f16", False, 9, 1, 127, 16), ("f32", True, 4, 1, 66, 16)])
def test_decode_on_the_cuda_cores(dt, e4m3, H, Hkv, D, page):
    c = Cache(LENS, Hkv, D, page, DT[dt], e4m3, seed=H + D)
    q = torch.randn(len(LENS), H, D, generator=torch.Generator().manual_seed(2)).to(DT[dt])
    o, lse = decode(c, q)
    assert api.last_path() == 2
    check_decode(c, q, o, lse, D ** -0.5, False)


@pytest.mark.parametrize("dt,e4m3", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("lens", [[20000], [1, 9000, 3], [3000] * 3, [64] * 40, [1] * 200,
                                  [40] * 150 + [5000]])
def test_decode_split_over_long_contexts_and_many_sequences(dt, e4m3, lens):
    c = Cache(lens, 2, 64, 16, DT[dt], e4m3, seed=5)
    q = torch.randn(len(lens), 4, 64, generator=torch.Generator().manual_seed(4)).to(DT[dt])
    o, lse = decode(c, q)
    check_decode(c, q, o, lse, 0.125, dt != "f32")
    # the same call gives the same bits, also into a dirty workspace
    dev = c.cuda()
    need = api.decode_workspace_size(dev["k_cache"], dev["block_table"], 4, DT[dt])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        o2, lse2 = decode(c, q, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_scales(scale, e4m3):
    c = Cache([70, 5], 2, 64, 16, torch.float16, e4m3, seed=8)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(4)).half()
    o, lse = decode(c, q, scale=scale)
    check_decode(c, q, o, lse, scale, True)


@pytest.mark.parametrize("exp", [-100, -30, 30, 90])
def test_decode_over_e4m3_takes_any_magnitude(exp):
    """Queries, keys and values far from 1, so that fp16 alone would not hold them."""
    c = Cache([150, 20], 1, 64, 16, torch.bfloat16, True, seed=8)
    c.scales[0] = (c.scales[0].int() - exp).clamp(0, 247).to(torch.uint8)
    c.scales[1] = (c.scales[1].int() + exp).clamp(0, 247).to(torch.uint8)
    q = (torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(4)) * 2.0 ** exp).bfloat16()
    o, lse = decode(c, q)
    check_decode(c, q, o, lse, 0.125, True)


@pytest.mark.parametrize("dt,e4m3", [("bf16", False), ("f16", True), ("f32", False)])
def test_rows_behind_a_sequence_are_never_multiplied(dt, e4m3):
    """NaN and infinities in the unused rows of pages, and in unused pages."""
    lens = [1, 15, 33, 64, 90]
    c = Cache(lens, 2, 64, 16, DT[dt], e4m3, seed=11)
    q = torch.randn(len(lens), 4, 64, generator=torch.Generator().manual_seed(4)).to(DT[dt])
    want = decode(c, q)
    used = torch.zeros(c.pages, 16, dtype=torch.bool)
    for b, n in enumerate(lens):
        for r in range(n):
            used[int(c.table[b, r // 16]), r % 16] = True
    for x in (c.k, c.v):
        y = x.float()
        y.permute(0, 2, 1, 3)[~used] = float("nan")
        x.copy_(y.to(x.dtype))
    if e4m3:
        for s in c.scales:
            s.permute(0, 2, 1)[~used] = 255
    got = decode(c, q)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_special_values_among_the_keys():
    """A NaN key makes its row NaN and no other; logits of -inf drop out."""
    c = Cache([40, 40], 2, 64, 16, torch.bfloat16, False, seed=3)
    c.k[int(c.table[0, 1]), 1, 3, 5] = float("nan")  # sequence 0, head 1, position 19
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    o, lse = decode(c, q)
    assert torch.isnan(o[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.isfinite(o[0, :2]).all() and torch.isfinite(o[1]).all()


def test_bad_pages_and_lengths_are_skipped_and_reported():
    c = Cache([40, 64, 20], 2, 64, 16, torch.bfloat16, False, seed=3)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    c.table[0, 1] = c.pages  # positions 16..31 of sequence 0 are skipped
    c.table[1, 3] = -5
    o, lse = decode(c, q, lens=[40, 64, -3])
    assert api.device_status() == _abi.JVP_ERR_INDEX
    for b, keep in ((0, list(range(16)) + list(range(32, 40))), (1, list(range(48)))):
        t = c.table[b].clone()
        c.table[b] = torch.where((t < 0) | (t >= c.pages), 0, t)
        k, v = c.rows(b)
        for h in range(4):
            r = attend(f64(q[b, h])[None], k[h // 2][keep], v[h // 2][keep],
                       np.ones((1, len(keep)), bool), 0.125)
            b_o, b_lse = bounds(*r, 64, 64, 2.0 ** -8, 2.0 ** -8, True)
            assert (np.abs(f64(o[b, h]) - r[0][0]) <= b_o[0]).all()
            assert abs(f64(lse[b, h]) - r[1][0]) <= b_lse[0]
    assert o[2].eq(0).all() and torch.isneginf(lse[2]).all()
    # a length past the block table is taken as the table's
    o, _ = decode(c, q, lens=[40, 64, 10 ** 6])
    assert api.device_status() == _abi.JVP_ERR_INDEX
    assert torch.isfinite(o).all()


def test_strided_queries_outputs_and_caches():
    B, H, Hkv, D, page = 3, 4, 2, 64, 16
    lens = [33, 5, 64]
    c = Cache(lens, Hkv, D, page, torch.float16, False, seed=6)
    dev = c.cuda()
    both = torch.stack([dev["k_cache"].transpose(1, 2), dev["v_cache"].transpose(1, 2)], 2).contiguous()
    kc, vc = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    wide = torch.randn(B, 3 * H, D, generator=torch.Generator().manual_seed(4)).half().cuda()
    q = wide[:, H:2 * H]
    out = torch.full((H, B, D + 8), 9.0, device="cuda", dtype=torch.float16)
    o = out.transpose(0, 1)[..., :D]
    table = torch.full((B, 9), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = dev["block_table"]
    r, lse = api.attention_decode(q, kc, vc, table[:, :c.table.shape[1]], i32(lens), out=o,
                                  return_lse=True)
    assert r is o and api.last_path() == 1
    check_decode(c, q.cpu(), o, lse, D ** -0.5, True)
    assert out[..., D:].eq(9.0).all()
    # rows that are not 16-byte aligned take the CUDA cores
    off = torch.zeros(c.pages, Hkv, page, D + 1, device="cuda", dtype=torch.float16)
    off2 = torch.zeros_like(off)
    off[..., 1:], off2[..., 1:] = dev["k_cache"], dev["v_cache"]
    r, lse = api.attention_decode(q, off[..., 1:], off2[..., 1:], dev["block_table"], i32(lens),
                                  return_lse=True)
    assert api.last_path() == 2
    check_decode(c, q.cpu(), r, lse, D ** -0.5, False)


def test_offsets_past_32_bits():
    """Pages further apart than 2^32 elements: 9 GB caches of which three pages are used."""
    D, Hkv, page = 128, 1, 16
    far = (1 << 32) // (page * D) + 3  # this page starts past element 2^32
    kc = torch.empty(far + 1, Hkv, page, D, dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.empty_like(kc)
    ks, vs = (torch.empty(far + 1, Hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2))
    T = 40
    table = i32([[far, 2, far - 1]])
    k, v = (torch.randn(T, Hkv, D, device="cuda").bfloat16() for _ in range(2))
    api.cache_write(k, v, kc, vc, table, None, cu_of([T]), k_scale=ks, v_scale=vs)
    rk, rv = api.cache_read(kc, vc, table, None, cu_of([T]), num_rows=T, k_scale=ks, v_scale=vs)
    for x, y in ((k, rk), (v, rv)):
        codes, e = quantise(f64(x))
        np.testing.assert_array_equal(f64(y), codes * np.exp2(e)[..., None])
    q = torch.randn(1, 4, D, device="cuda").bfloat16()
    o, lse = api.attention_decode(q, kc, vc, table, i32([T]), k_scale=ks, v_scale=vs, return_lse=True)
    for h in range(4):
        r = attend(f64(q[0, h])[None], f64(rk[:, 0]), f64(rv[:, 0]), np.ones((1, T), bool), D ** -0.5)
        b_o, b_lse = bounds(*r, T, D, 2.0 ** -8, 2.0 ** -11, True)
        assert (np.abs(f64(o[0, h]) - r[0][0]) <= b_o[0]).all()


def test_decode_on_another_stream_and_in_a_graph_that_follows_the_lengths():
    lens = [100, 31]
    c = Cache([200, 200], 2, 64, 16, torch.bfloat16, True, seed=12)
    dev = c.cuda()
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    dq, dl = q.cuda(), i32(lens)
    k, v = (torch.randn(2, 2, 64, device="cuda").bfloat16() for _ in range(2))
    out = torch.empty_like(dq)

    def step():  # a decoding step: the token's row in, attention over it
        api.cache_write(k, v, dev["k_cache"], dev["v_cache"], dev["block_table"], dl,
                        k_scale=dev["k_scale"], v_scale=dev["v_scale"])
        dl.add_(1)
        return api.attention_decode(dq, dev["k_cache"], dev["v_cache"], dev["block_table"], dl,
                                    k_scale=dev["k_scale"], v_scale=dev["v_scale"], out=out,
                                    return_lse=True)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    codes = [quantise(f64(x)) for x in (k, v)]
    for n in range(2, 5):
        graph.replay()
        torch.cuda.synchronize()
        now = [x + n for x in lens]
        for b in range(2):
            for pos in range(lens[b], now[b]):
                pg, r = int(c.table[b, pos // 16]), pos % 16
                for i, t in enumerate((c.k, c.v)):
                    t[pg, :, r] = torch.from_numpy(codes[i][0][b]).to(torch.float8_e4m3fn)
                    c.scales[i][pg, :, r] = torch.from_numpy(codes[i][1][b] + 127).to(torch.uint8)
        check_decode(c, q, o, lse, 0.125, True, lens=now)


def test_decode_joins_a_dense_cache_read():
    """Reading the cache back and running the dense attention gives the same."""
    lens = [77]
    c = Cache(lens, 2, 64, 16, torch.bfloat16, True, seed=12)
    dev = c.cuda()
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    o, lse = decode(c, q)
    k, v = api.cache_read(dev["k_cache"], dev["v_cache"], dev["block_table"], None, cu_of(lens),
                          num_rows=77, k_scale=dev["k_scale"], v_scale=dev["v_scale"])
    dense, dl = api.attention(q.view(1, 4, 1, 64), k.transpose(0, 1)[None], v.transpose(0, 1)[None],
                              return_lse=True)
    check_decode(c, q, dense.view(1, 4, 64), dl.view(1, 4), 0.125, True)
    check_decode(c, q, o, lse, 0.125, True)


def test_empty_problems():
    kc = torch.zeros(4, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    t0 = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    o, lse = api.attention_decode(torch.zeros(0, 4, 64, device="cuda", dtype=torch.bfloat16), kc, kc,
                                  t0, i32([]), return_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    # no pages at all: empty rows
    none = torch.zeros(0, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    q = torch.ones(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    for table in (torch.zeros(2, 0, dtype=torch.int32, device="cuda"), i32([[-1], [-1]])):
        o, lse = api.attention_decode(q, none, none, table, i32([0, 0]), return_lse=True)
        assert o.eq(0).all() and torch.isneginf(lse).all()
    e = torch.zeros(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    api.cache_write(e, e, kc, kc.clone(), i32([[0], [1]]), None, i32([0, 0, 0]))
    assert kc.eq(0).all()
    k, v = api.cache_read(kc, kc, i32([[0]]), None, i32([0, 0]), num_rows=0)
    assert k.shape == (0, 2, 64)


@pytest.mark.parametrize("e4m3", [False, True])
def test_split_decode_in_graphs_that_follow_the_lengths(e4m3):
    """Long block tables, so that segments are split and combined: two captured
    calls, replayed with other lengths, beside eager calls on another stream."""
    B, most = 5, 9000
    c = Cache([most] * B, 2, 64, 16, torch.bfloat16, e4m3, seed=13)
    dev = c.cuda()
    q = torch.randn(B, 4, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    dq, dl = q.cuda(), i32([most] * B)

    def call(lens, **kw):
        return api.attention_decode(dq, dev["k_cache"], dev["v_cache"], dev["block_table"], lens,
                                    k_scale=dev["k_scale"], v_scale=dev["v_scale"], return_lse=True, **kw)

    want = {}
    for lens in ([most, 0, 70, 1, 5000], [0, 0, 0, 0, most], [0] * 5, [most] * 5):
        want[tuple(lens)] = call(i32(lens))
        check_decode(c, q, *want[tuple(lens)], 0.125, True, lens=lens)
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(dl))
        graphs.append(g)
    fixed = i32([3000, 1, most, 0, 2])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        alone = call(fixed)
    side.synchronize()
    for lens, (o, lse) in want.items():
        dl.copy_(i32(list(lens)))
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            with torch.cuda.stream(side):
                o2, lse2 = call(fixed)
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, alone[0]) and torch.equal(lse2, alone[1])
        for og, lg in outs:
            assert torch.equal(og, o) and torch.equal(lg, lse)
