"""Attention of chunks of new tokens over a paged cache, with and without a window,
against the definition in float64 (bounds derived in serving_ref.py)."""

import numpy as np
import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build
from serving_ref import Cache, attend, bounds, f64

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


def make(new, past, H, Hkv, D, dt, page=16, e4m3=False, seed=0, before=0, behind=0):
    """A cache with past + new rows of each sequence, queries, offsets."""
    total = [max(0, a + b) for a, b in zip(new, past)]
    c = Cache(total, Hkv, D, page, DT[dt], e4m3, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(before + sum(new) + behind, H, D, generator=g).to(DT[dt])
    cu = torch.tensor(before + np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return c, q, cu


def run(c, q, cu, window=None, sinks=0, lens=None, **kw):
    d = c.cuda()
    lens = torch.tensor(c.lens if lens is None else lens, dtype=torch.int32).cuda()
    return api.attention_chunk(q.cuda(), d["k_cache"], d["v_cache"], d["block_table"], lens, cu.cuda(),
                               window=window, sinks=sinks, k_scale=d["k_scale"], v_scale=d["v_scale"],
                               return_lse=True, **kw)


def check(c, q, cu, o, lse, window=None, sinks=0, scale=None, heads=None, rows=None):
    T, H, D = q.shape
    G = H // c.Hkv
    tc = api.last_path() == 1
    u = torch.finfo(q.dtype).eps / 2
    w = u if tc else 0.0
    scale = D ** -0.5 if scale is None else scale
    o, lse = f64(o), f64(lse)
    for b, n in enumerate(c.lens):
        r = np.arange(int(cu[b]), int(cu[b + 1]))
        x = n - len(r) + np.arange(len(r))  # positions
        if rows is not None and len(r) > rows:
            some = np.unique(np.linspace(0, len(r) - 1, rows).astype(int))
            r, x = r[some], x[some]
        if len(r) == 0:
            continue
        k, v = c.rows(b)
        if c.e4m3 and tc and q.dtype == torch.float16:  # taken as cache_read gives them
            k, v = k.astype(np.float16).astype(np.float64), v.astype(np.float16).astype(np.float64)
        j = np.arange(n)
        keep = j <= x[:, None]
        if window is not None:
            keep &= (j > x[:, None] - window) | (j < sinks)
        for h in (range(H) if heads is None else heads):
            ref = attend(f64(q[r, h]), k[h // G], v[h // G], keep, scale)
            b_o, b_lse = bounds(*ref, max(n, 1), D, u, w, tc)
            e = np.abs(o[r, h] - ref[0])
            assert (e <= b_o).all(), (b, h, np.unravel_index((e - b_o).argmax(), e.shape), e.max())
            none = np.isneginf(ref[1])
            assert np.isneginf(lse[h, r][none]).all(), (b, h)
            assert (np.abs(lse[h, r] - ref[1])[~none] <= b_lse[~none]).all(), (b, h)


NEW = [1, 0, 7, 33, 128, 200, 2, 65]
PAST = [0, 5, 120, 300, 1, 0, 700, 127]
SHAPES = [("bf16", 8, 2, 128, 16), ("f16", 4, 4, 64, 32), ("bf16", 16, 1, 64, 8), ("f16", 3, 1, 128, 128),
          ("bf16", 12, 4, 40, 24), ("f16", 5, 5, 96, 64), ("bf16", 6, 2, 80, 48), ("bf16", 7, 1, 8, 256)]


@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (50, 3), (128, 0), (200, 130), (300, 1)])
@pytest.mark.parametrize("dt,H,Hkv,D,page", SHAPES)
def test_ragged_chunks_on_the_tensor_cores(dt, H, Hkv, D, page, window, sinks):
    c, q, cu = make(NEW, PAST, H, Hkv, D, dt, page, seed=D)
    o, lse = run(c, q, cu, window, sinks)
    assert api.last_path() == 1
    check(c, q, cu, o, lse, window, sinks, heads=sorted({0, H // 2, H - 1}))


GATHERED = [("bf16", 8, 2, 128, 16, True), ("f16", 4, 4, 64, 32, True), ("bf16", 16, 1, 64, 1, True),
            ("f16", 3, 1, 128, 100, True), ("bf16", 12, 4, 40, 24, True), ("bf16", 7, 1, 8, 3, True),
            ("bf16", 8, 2, 128, 1, False), ("f16", 4, 4, 64, 20, False), ("bf16", 5, 5, 96, 7, False),
            ("f16", 12, 4, 40, 130, False)]


@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (50, 3), (200, 130)])
@pytest.mark.parametrize("dt,H,Hkv,D,page,e4m3", GATHERED)
def test_gathered_rows(dt, H, Hkv, D, page, e4m3, window, sinks):
    """e4m3 caches, and pages that are no multiple of 8 rows."""
    c, q, cu = make(NEW, PAST, H, Hkv, D, dt, page, e4m3, seed=D)
    o, lse = run(c, q, cu, window, sinks)
    assert api.last_path() == 1
    check(c, q, cu, o, lse, window, sinks, heads=sorted({0, H // 2, H - 1}))


@pytest.mark.parametrize("dt,H,Hkv,D,page,e4m3", [("bf16", 8, 2, 128, 16, True), ("f16", 2, 2, 64, 5, False),
                                                  ("f16", 4, 1, 64, 64, True)])
@pytest.mark.parametrize("new,past", [([1700], [900]), ([3] * 90, [40] * 90), ([4, 1, 70], [9000, 20000, 5000])],
                         ids=["one", "ninety", "split"])
def test_gathered_rows_of_long_chunks_and_contexts(new, past, dt, H, Hkv, D, page, e4m3):
    c, q, cu = make(new, past, H, Hkv, D, dt, page, e4m3, seed=4)
    o, lse = run(c, q, cu)
    assert api.last_path() == 1
    check(c, q, cu, o, lse, heads=[0, H - 1], rows=60)
    o2, lse2 = run(c, q, cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 1), (50, 3), (200, 70)])
@pytest.mark.parametrize("dt,H,Hkv,D,page,e4m3", [
    ("f32", 4, 2, 64, 16, False), ("f32", 2, 2, 128, 7, False), ("f32", 3, 1, 33, 1, False),
    ("bf16", 4, 1, 20, 16, False), ("f16", 2, 1, 127, 24, False), ("f32", 4, 2, 64, 16, True),
    ("f32", 40, 1, 16, 16, False), ("f32", 2, 1, 30, 5, True)])
def test_ragged_chunks_on_the_cuda_cores(dt, H, Hkv, D, page, e4m3, window, sinks):
    c, q, cu = make(NEW, PAST, H, Hkv, D, dt, page, e4m3, seed=D)
    o, lse = run(c, q, cu, window, sinks)
    assert api.last_path() == 2
    check(c, q, cu, o, lse, window, sinks, heads=sorted({0, H // 2, H - 1}))


@pytest.mark.parametrize("window,sinks", [(None, 0), (100, 5), (900, 0)])
@pytest.mark.parametrize("dt,H,Hkv,D", [("bf16", 4, 1, 128), ("f16", 2, 2, 64), ("f32", 2, 1, 64)])
@pytest.mark.parametrize("new,past", [
    ([1700], [900]), ([900, 1, 1100], [0, 2500, 333]), ([3] * 90, [40] * 90),
    ([1] * 300, list(range(300))), ([300] * 12, [128] * 12)],
    ids=["one", "three", "ninety", "tokens", "twelve"])
def test_long_chunks_and_many_sequences(new, past, dt, H, Hkv, D, window, sinks):
    c, q, cu = make(new, past, H, Hkv, D, dt, seed=3)
    o, lse = run(c, q, cu, window, sinks)
    check(c, q, cu, o, lse, window, sinks, heads=[0, H - 1], rows=60)
    o2, lse2 = run(c, q, cu, window, sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window,sinks", [(None, 0), (3000, 200)])
@pytest.mark.parametrize("dt,H,Hkv,D", [("bf16", 8, 2, 128), ("f16", 4, 4, 64), ("f32", 4, 2, 64)])
def test_few_tokens_over_long_contexts_are_split(dt, H, Hkv, D, window, sinks):
    c, q, cu = make([4, 1, 70], [9000, 20000, 5000], H, Hkv, D, dt, 64, seed=6)
    o, lse = run(c, q, cu, window, sinks)
    check(c, q, cu, o, lse, window, sinks, heads=[0, H - 1])
    o2, lse2 = run(c, q, cu, window, sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_sequences_of_few_tokens_over_long_contexts(dt):
    """More sequences than lanes of a warp, some of them cut."""
    past = [10 + 61 * i for i in range(70)]
    past[13], past[50] = 16000, 0
    c, q, cu = make([2] * 70, past, 4, 2, 64, dt, 32, seed=8)
    o, lse = run(c, q, cu)
    check(c, q, cu, o, lse, heads=[0, 3])


@pytest.mark.parametrize("dt,page", [("bf16", 16), ("f16", 5), ("f32", 16)])
def test_thousands_of_sequences(dt, page):
    """More than the division holds at a time, some of no tokens, one long one among them."""
    new = [(0, 1, 3, 0, 2)[i % 5] for i in range(5003)]
    past = [(7 * i) % 41 for i in range(5003)]
    new[3100], past[3100] = 700, 5000
    c, q, cu = make(new, past, 2, 1, 64, dt, page, seed=17)
    o, lse = run(c, q, cu)
    check(c, q, cu, o, lse, heads=[1], rows=40)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_whole_prompts_agree_with_packed_attention(dt):
    """Chunks without a past are packed prompts (same definition, same bounds)."""
    new = [300, 17, 1, 640]
    c, q, cu = make(new, [0] * 4, 4, 2, 64, dt, seed=11)
    o, lse = run(c, q, cu)
    check(c, q, cu, o, lse)
    d = c.cuda()
    k, v = api.cache_read(d["k_cache"], d["v_cache"], d["block_table"], None, cu.cuda(), num_rows=sum(new))
    p, plse = api.attention_packed(q.cuda(), k, v, cu.cuda(), is_causal=True, return_lse=True)
    fake = type("C", (), {})()
    fake.lens, fake.Hkv, fake.e4m3, fake.rows = c.lens, c.Hkv, False, c.rows
    check(fake, q, cu, p, plse)


@pytest.mark.parametrize("dt", ["bf16", "f32", "e4m3"])
def test_tokens_before_the_first_position_see_nothing(dt):
    c, q, cu = make([5, 200, 3], [-2, -190, -3], 4, 2, 64, "bf16" if dt == "e4m3" else dt,
                    e4m3=dt == "e4m3", seed=2)
    assert c.lens == [3, 10, 0]
    o, lse = run(c, q, cu)
    check(c, q, cu, o, lse)
    assert (o[:2] == 0).all() and torch.isneginf(lse[:, :2]).all()
    assert (o[-3:] == 0).all() and torch.isneginf(lse[:, -3:]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_padded_batch_leaves_its_other_rows(dt):
    c, q, cu = make([30, 1], [3, 99], 4, 2, 64, dt, seed=2, before=6, behind=9)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    o, lse = run(c, q, cu, out=out)
    assert o.data_ptr() == out.data_ptr()
    assert (o[:6] == 7).all() and (o[-9:] == 7).all()
    check(c, q, cu, o, lse)


@pytest.mark.parametrize("window,sinks", [(None, 0), (70, 3), (300, 140)])
@pytest.mark.parametrize("dt,page,e4m3", [
    ("bf16", 16, False), ("f16", 64, False), ("f32", 16, False), ("bf16", 8, False), ("f16", 20, False),
    ("bf16", 16, True), ("f16", 7, True), ("f32", 16, True)])
def test_what_rows_do_not_see_has_no_say(dt, page, e4m3, window, sinks):
    """Infinities and NaN at later positions, before the window and behind the end
    (in the last page) change nothing; pages that no token sees need not exist."""
    new, past = [40, 3, 130], [500, 700, 333]
    c, q, cu = make(new, past, 4, 2, 64, dt, page, e4m3, seed=5)
    want = run(c, q, cu, window, sinks)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan")]).repeat(16)
    if e4m3:  # (codes hold NaN but no infinities)
        bad = torch.full((64,), float("nan"))
    some = torch.ones(len(q), dtype=torch.bool)
    for b, n in enumerate(c.lens):
        place = lambda j: (int(c.table[b, j // page]), j % page)  # noqa: E731
        first = n - new[b]
        hide = list(range(sinks, first - window + 1)) if window else []
        for j in hide + list(range(n, -(-n // page) * page)):
            pg, r = place(j)
            c.k[pg, :, r] = bad.to(c.k.dtype)
            c.v[pg, :, r] = bad.flip(0).to(c.v.dtype)
        # the last two new rows: only the last two tokens see them
        for j in (n - 2, n - 1):
            pg, r = place(j)
            c.v[pg, :, r] = bad.to(c.v.dtype)
        some[int(cu[b + 1]) - 2:int(cu[b + 1])] = False
        if window:
            # a row that leaves the window inside the chunk: later tokens do not see it
            j = first - window + 1 + new[b] // 2
            if j >= sinks:
                pg, r = place(j)
                c.v[pg, :, r] = bad.to(c.v.dtype)
                x = first + np.arange(new[b])
                some[int(cu[b]):int(cu[b + 1])] &= torch.from_numpy(x - window >= j)
            for e in range(-(-sinks // page), max(0, first - window + 1) // page):
                c.table[b, e] = -9
    assert some.any()
    got = run(c, q, cu, window, sinks)
    some = some.cuda()
    assert torch.equal(got[0][some], want[0][some])
    assert torch.equal(got[1][:, some], want[1][:, some])
    # and the rows that do see them hold what the definition gives: NaN and infinities
    last = got[0][int(cu[1]) - 1].float().cpu()
    if e4m3:
        assert torch.isnan(last).all()
        return
    assert torch.isnan(last[:, 0]).all() and (last[:, 1] == float("inf")).all()
    assert (last[:, 2] == -float("inf")).all()


@pytest.mark.parametrize("dt,e4m3", [("bf16", False), ("f32", False), ("bf16", True)])
def test_pages_that_do_not_exist_are_skipped_and_reported(dt, e4m3):
    c, q, cu = make([5, 3], [300, 40], 4, 2, 64, dt, e4m3=e4m3, seed=5)
    c.table[0, 4] = c.pages          # positions 64 .. 79 of the first
    c.table[0, 19] = -3              # its last page: positions 304 and on
    got = run(c, q, cu)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    ok = np.array([j // 16 not in (4, 19) for j in range(305)])
    c.table[0, 4] = c.table[0, 19] = 0
    k, v = c.rows(0)
    x = 300 + np.arange(5)
    keep = (np.arange(305) <= x[:, None]) & ok
    tc = api.last_path() == 1
    u = torch.finfo(q.dtype).eps / 2
    for h in range(4):
        ref = attend(f64(q[:5, h]), k[h // 2], v[h // 2], keep, 64 ** -0.5)
        b_o, b_lse = bounds(*ref, 305, 64, u, u if tc else 0.0, tc)
        assert (np.abs(f64(got[0])[:5, h] - ref[0]) <= b_o).all()
        assert (np.abs(f64(got[1])[h, :5] - ref[1]) <= b_lse).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_bad_offsets_and_lengths_are_reported(dt):
    c, q, cu = make([5, 3, 4], [30, 40, 0], 4, 2, 64, dt, seed=5)
    good = run(c, q, cu)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    run(c, q, torch.tensor([0, 5, 3, 12], dtype=torch.int32), out=out)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    assert torch.equal(out[:3], good[0][:3])  # (rows 3 and 4 are in the third sequence too)
    out.fill_(7.0)
    run(c, q, torch.tensor([0, 5, 8, 13], dtype=torch.int32), out=out)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    assert (out[8:] == 7).all() and torch.equal(out[:8], good[0][:8])
    run(c, q, cu, lens=[35, 43, 100000])
    assert api.device_status() == _abi.JVP_ERR_INDEX
    run(c, q, cu, lens=[35, 43, -1])
    assert api.device_status() == _abi.JVP_ERR_INDEX


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_scales(dt, scale):
    c, q, cu = make([200, 9], [50, 400], 4, 2, 64, dt, seed=5)
    o, lse = run(c, q, cu, 120, 2, scale=scale)
    assert api.last_path() == (1 if dt == "f16" and scale != 0 else 2)
    check(c, q, cu, o, lse, 120, 2, scale=scale)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_alignment(dt):
    """Queries and outputs inside wider rows, a cache with heads behind rows, rows off their
    alignment."""
    c, q, cu = make([20, 140], [300, 5], 4, 2, 64, dt, seed=7)
    want = run(c, q, cu)
    d = c.cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    wide = torch.zeros(len(q), 12, 64, dtype=q.dtype, device="cuda")
    wide[:, 4:8] = q.cuda()
    out = torch.zeros_like(wide)
    o = api.attention_chunk(wide[:, 4:8], d["k_cache"], d["v_cache"], d["block_table"], lens, cu.cuda(),
                            out=out[:, 8:])
    assert torch.equal(o, want[0]) and (out[:, :8] == 0).all()
    by_row = [d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("k_cache", "v_cache")]
    o = api.attention_chunk(q.cuda(), *by_row, d["block_table"], lens, cu.cuda())
    assert torch.equal(o, want[0])
    odd = []
    for n in ("k_cache", "v_cache"):
        x = torch.zeros(*d[n].shape[:3], 65, dtype=q.dtype, device="cuda")[..., 1:]
        x.copy_(d[n])
        odd.append(x)
    o, lse = api.attention_chunk(q.cuda(), *odd, d["block_table"], lens, cu.cuda(), return_lse=True)
    check(c, q, cu, o, lse)


def test_captured_graph_follows_lengths():
    c, q, cu = make([4, 60, 30], [2000, 100, 700], 8, 2, 128, "bf16", seed=9)
    d, qc = c.cuda(), q.cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    off = cu.cuda()
    args = (qc, d["k_cache"], d["v_cache"], d["block_table"], lens, off)
    api.attention_chunk(*args, window=500, sinks=4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = api.attention_chunk(*args, window=500, sinks=4)
    lens.copy_(torch.tensor([700, 160, 730], dtype=torch.int32))
    off.copy_(torch.tensor([0, 70, 70, 94], dtype=torch.int32))
    graph.replay()
    assert torch.equal(o, api.attention_chunk(*args, window=500, sinks=4))


def test_a_workspace_and_two_streams():
    c, q, cu = make([4, 1], [9000, 20000], 8, 2, 128, "bf16", 64, seed=9)
    want = run(c, q, cu)
    d = c.cuda()
    need = api.chunk_workspace_size(q.cuda(), d["k_cache"], d["block_table"])
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = run(c, q, cu, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(_abi.JvpAttnError):
        run(c, q, cu, workspace=ws[:1024])
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    args = (q.cuda(), d["k_cache"], d["v_cache"], d["block_table"], lens, cu.cuda())
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            outs.append(api.attention_chunk(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) for o in outs)


def test_values_of_an_e4m3_cache_that_fp16_cannot_hold():
    """Taken as cache_read gives them: infinite above 65504, multiples of 2^-24 below."""
    c, q, cu = make([3], [40], 2, 1, 64, "f16", e4m3=True, seed=2)
    c.scales[1][:] = 127 + 12
    o, lse = run(c, q, cu)
    d = c.cuda()
    k, v = api.cache_read(d["k_cache"], d["v_cache"], d["block_table"], None,
                          torch.tensor([0, 43], dtype=torch.int32).cuda(), num_rows=43,
                          k_scale=d["k_scale"], v_scale=d["v_scale"], dtype=torch.float16)
    big = torch.isinf(v[:41, 0])  # seen by every token
    assert big.any()
    assert not torch.isfinite(o[:, :, big.any(0)]).any()
    c.scales[1][:] = 127 - 20
    c.scales[0][:] = 127 - 24
    o, lse = run(c, q, cu)
    check(c, q, cu, o, lse)


def test_no_rows():
    c, q, cu = make([0, 0], [3, 4], 4, 2, 64, "bf16", seed=1)
    o, lse = run(c, q, cu)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    c, q, cu = make([0, 2, 0], [3, 4, 9], 4, 2, 64, "bf16", seed=1)
    o, lse = run(c, q, cu)
    check(c, q, cu, o, lse)


def test_refusals():
    c, q, cu = make([2], [4], 4, 2, 64, "bf16", seed=1)
    for kw in (dict(window=0), dict(window=-3), dict(window=4, sinks=-1),
               dict(workspace=torch.empty(4, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            run(c, q, cu, **kw)
    for bad in (q[:, :3], q.float(), q[..., :32], q[0]):
        with pytest.raises((ValueError, TypeError)):
            run(c, bad, cu)
    for bad in (cu.long(), cu[:1], cu[None]):
        with pytest.raises(ValueError):
            run(c, q, bad)
    with pytest.raises(_abi.JvpAttnError):
        run(c, q, cu, scale=float("nan"))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("page", [16, 5])
def test_every_code_of_an_e4m3_cache(dt, page):
    """A sequence of one key returns its values: all 256 codes under scales from the
    smallest to the largest, as cache_read gives them (NaN included)."""
    D, n = 128, 254
    c, q, cu = make([1] * n, [0] * n, 2, 2, D, dt, page, True, seed=3)
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8)
    c.k.view(torch.uint8).zero_()
    for b in range(n):
        pg = int(c.table[b, 0])
        c.v.view(torch.uint8)[pg, :, 0] = codes.view(2, D)
        c.scales[1][pg, :, 0] = b  # 2^-127 .. 2^126
    o, lse = run(c, q, cu)
    assert api.last_path() == 1
    d = c.cuda()
    _, v = api.cache_read(d["k_cache"], d["v_cache"], d["block_table"], None, cu.cuda(), num_rows=n,
                          k_scale=d["k_scale"], v_scale=d["v_scale"], dtype=DT[dt])
    same = (o == v) | (torch.isnan(o) & torch.isnan(v))
    assert same.all(), same.logical_not().nonzero()[:5]


@pytest.mark.parametrize("window,sinks", [(5, 900), (5, 2 ** 40), (2 ** 40, 7), (130, 128), (128, 129)])
@pytest.mark.parametrize("dt,H,Hkv,D,page,e4m3", [
    ("bf16", 8, 2, 128, 16, False), ("f16", 4, 4, 64, 20, False), ("bf16", 8, 2, 128, 16, True),
    ("f32", 4, 2, 64, 16, False)])
def test_sinks_that_reach_into_the_window(dt, H, Hkv, D, page, e4m3, window, sinks):
    c, q, cu = make(NEW, PAST, H, Hkv, D, dt, page, e4m3, seed=D + 1)
    o, lse = run(c, q, cu, window, sinks)
    check(c, q, cu, o, lse, window, sinks, heads=[0, H - 1])


@pytest.mark.parametrize("dt,e4m3", [("bf16", False), ("bf16", True), ("f32", False)])
def test_sequences_that_share_pages(dt, e4m3):
    """A common beginning, cached once: each sequence as by itself."""
    c, q, cu = make([40, 40, 3], [600, 600, 600], 4, 2, 64, dt, 16, e4m3, seed=9)
    c.table[1:, :40] = c.table[0, :40]  # (the last pages are each one's own)
    o, lse = run(c, q, cu)
    check(c, q, cu, o, lse)
