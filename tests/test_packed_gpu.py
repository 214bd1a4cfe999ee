"""Attention over packed prompts against the definition in float64 (bounds
derived in serving_ref.py)."""

import numpy as np
import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build
from serving_ref import attend, bounds, f64

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


def make(lens, H, Hkv, D, dt, seed=0, before=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    T = before + sum(lens) + behind
    q, k, v = (torch.randn(T, h, D, generator=g).to(DT[dt]) for h in (H, Hkv, Hkv))
    cu = torch.tensor(before + np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return q, k, v, cu


def check(q, k, v, cu, causal, o, lse, scale=None, tensor_cores=True, heads=None):
    T, H, D = q.shape
    G = H // k.shape[1]
    u = torch.finfo(q.dtype).eps / 2
    w = u if tensor_cores else 0.0
    scale = D ** -0.5 if scale is None else scale
    o, lse = f64(o), f64(lse)
    for b in range(len(cu) - 1):
        r = slice(int(cu[b]), int(cu[b + 1]))
        n = r.stop - r.start
        if n == 0:
            continue
        keep = np.tril(np.ones((n, n), bool)) if causal else np.ones((n, n), bool)
        for h in (range(H) if heads is None else heads):
            ref = attend(f64(q[r, h]), f64(k[r, h // G]), f64(v[r, h // G]), keep, scale)
            b_o, b_lse = bounds(*ref, n, D, u, w, tensor_cores)
            e = np.abs(o[r, h] - ref[0])
            assert (e <= b_o).all(), (b, h, np.unravel_index((e - b_o).argmax(), e.shape), e.max())
            assert (np.abs(lse[h, r] - ref[1]) <= b_lse).all(), (b, h)


def run(q, k, v, cu, causal, **kw):
    return api.attention_packed(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), is_causal=causal,
                                return_lse=True, **kw)


LENS = [1, 0, 2, 127, 128, 129, 5, 255, 256, 257, 0, 33, 400]
# long on average: two query tiles per CTA
LONG = [1025, 900, 1, 1281, 1152, 1300]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [LENS, LONG], ids=["short", "long"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hkv,D", [(2, 2, 128), (2, 2, 64), (8, 2, 128), (16, 1, 64), (3, 1, 128),
                                     (7, 1, 64), (5, 5, 96), (12, 4, 40), (40, 1, 8), (6, 2, 80)])
def test_ragged_prompts_on_the_tensor_cores(H, Hkv, D, dt, causal, lens):
    q, k, v, cu = make(lens, H, Hkv, D, dt, seed=H + D)
    o, lse = run(q, k, v, cu, causal)
    assert api.last_path() == 1
    check(q, k, v, cu, causal, o, lse, heads=None if lens is LENS else sorted({0, H // 2, H - 1}))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt,H,Hkv,D", [("f32", 2, 2, 64), ("f32", 4, 1, 128), ("f32", 2, 2, 33),
                                        ("bf16", 4, 2, 20), ("f16", 3, 3, 1), ("f32", 2, 1, 100),
                                        ("f16", 2, 2, 127)])
def test_ragged_prompts_on_the_cuda_cores(dt, H, Hkv, D, causal):
    q, k, v, cu = make(LENS, H, Hkv, D, dt, seed=H + D)
    o, lse = run(q, k, v, cu, causal)
    assert api.last_path() == 2
    check(q, k, v, cu, causal, o, lse, tensor_cores=False)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt,H,Hkv,D", [("bf16", 4, 1, 128), ("f16", 2, 2, 64), ("f32", 1, 1, 64)])
@pytest.mark.parametrize("lens", [[3001], [1500, 1, 1400], [7] * 90, [1] * 300, [300] * 12])
def test_long_prompts_and_many_prompts(lens, dt, H, Hkv, D, causal):
    q, k, v, cu = make(lens, H, Hkv, D, dt, seed=3)
    o, lse = run(q, k, v, cu, causal)
    check(q, k, v, cu, causal, o, lse, tensor_cores=dt != "f32", heads=[0, H - 1])
    o2, lse2 = run(q, k, v, cu, causal)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_heads_wider_than_a_tile(dt):
    """More query heads per key/value head than a tile has rows."""
    q, k, v, cu = make([3, 70], 130, 1, 16, dt, seed=3)
    o, lse = run(q, k, v, cu, True)
    assert api.last_path() == 2
    check(q, k, v, cu, True, o, lse, tensor_cores=False, heads=[0, 64, 129])
    q, k, v, cu = make([3, 70], 128, 1, 16, dt, seed=3)
    o, lse = run(q, k, v, cu, True)
    check(q, k, v, cu, True, o, lse, tensor_cores=dt == "bf16", heads=[0, 64, 127])


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_scales(dt, scale):
    q, k, v, cu = make([200, 9], 4, 2, 64, dt, seed=5)
    o, lse = run(q, k, v, cu, True, scale=scale)
    assert api.last_path() == (1 if dt == "f16" and scale != 0 else 2)
    check(q, k, v, cu, True, o, lse, scale=scale, tensor_cores=api.last_path() == 1)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_large_logits_move_the_running_maximum(dt):
    """Keys that grow along the sequence: every tile rescales what came before."""
    q, k, v, cu = make([700, 300], 2, 1, 64, dt, seed=6)
    ramp = torch.linspace(0.2, 6.0, len(k))[:, None, None]
    q, k = (q.abs() * 2).to(DT[dt]), (k.abs() * ramp).to(DT[dt])
    for causal in (False, True):
        o, lse = run(q, k, v, cu, causal)
        check(q, k, v, cu, causal, o, lse, tensor_cores=dt != "f32")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[130, 60, 200], [1100, 790, 900]], ids=["short", "long"])
@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("f32", 64)])
def test_rows_of_other_sequences_and_of_none_have_no_say(dt, D, causal, lens):
    """NaN and infinities in the rows around the sequences; those rows stay as they were."""
    H, Hkv = 4, 2
    q, k, v, cu = make(lens, H, Hkv, D, dt, seed=7, before=3, behind=50)
    want, wl = run(q, k, v, cu, causal)
    check(q, k, v, cu, causal, want, wl, tensor_cores=dt != "f32", heads=[0, 3])
    inside = torch.zeros(len(q), dtype=torch.bool)
    inside[3:3 + sum(lens)] = True
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[~inside] = bad
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    o, lse = run(q, k, v, cu, causal, out=out)
    assert o is out
    assert torch.equal(o[inside.cuda()], want[inside.cuda()])
    assert torch.equal(lse[:, inside.cuda()], wl[:, inside.cuda()])
    assert out[~inside.cuda()].eq(5.0).all()
    # a sequence full of NaN between two others
    r = slice(int(cu[1]), int(cu[2]))
    k[r], v[r] = float("nan"), float("inf")
    o, _ = run(q, k, v, cu, causal)
    for b in (0, 2):
        s = slice(int(cu[b]), int(cu[b + 1]))
        assert torch.equal(o[s], want[s])
    assert torch.isnan(o[r]).all()


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2)])
@pytest.mark.parametrize("lens", [[300, 5, 131], [1500, 1400]], ids=["short", "long"])
@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("f16", 40), ("f32", 64)])
def test_values_behind_a_row_have_no_say(dt, D, lens, H, Hkv):
    """Causal: infinities and NaN among later keys and values leave a row as it was; the rows
    that see them have them in the same columns."""
    q, k, v, cu = make(lens, H, Hkv, D, dt, seed=17)
    want, wl = run(q, k, v, cu, True)
    inf, nan = float("inf"), float("nan")
    places = [(lens[0] - 1, 0, 3, nan), (lens[0] - 150, Hkv - 1, D - 1, inf),
              (lens[0] // 2, 0, 0, -inf), (129, Hkv - 1, 17, inf), (130, Hkv - 1, 17, -inf),
              (0, 0, 5, inf), (lens[0] + 1, 0, 8, inf), (sum(lens) - 1, 0, 9, nan)]
    for row, h, d, x in places:
        v[row, h, d] = x
    o, lse = run(q, k, v, cu, True)
    expect = want.float().clone()
    ends = [int(e) for e in cu[1:]]
    for row, h, d, x in places:
        end = next(e for e in ends if row < e)
        heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
        expect[row:end, heads, d] += x
    bad = ~torch.isfinite(expect)
    assert bad.any() and not bad.all()
    assert torch.equal(o[~bad].float(), expect[~bad])
    assert torch.equal(torch.nan_to_num(o[bad].float(), nan=7.0),
                       torch.nan_to_num(expect[bad], nan=7.0))
    assert torch.equal(lse, wl)
    # keys too: the rows in front of a NaN key keep their bits
    row = lens[0] - 20
    k[row] = nan
    o2, _ = run(q, k, v, cu, True)
    same = o2[:row].eq(o[:row]) | (torch.isnan(o2[:row]) & torch.isnan(o[:row]))
    assert same.all()
    assert torch.isnan(o2[row:lens[0]]).all()


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f16", 128), ("f32", 64)])
def test_strides_of_a_joint_projection(dt, D):
    """q, k, v side by side in one tensor, the output into part of another."""
    T, H, Hkv = 150, 4, 2
    cu = torch.tensor([0, 100, 150], dtype=torch.int32)
    x = torch.randn(T, H + 2 * Hkv, D, generator=torch.Generator().manual_seed(1)).to(DT[dt]).cuda()
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    big = torch.full((T, 2 * H, D), 3.0, dtype=DT[dt], device="cuda")
    o, lse = api.attention_packed(q, k, v, cu.cuda(), is_causal=True, out=big[:, H:], return_lse=True)
    assert api.last_path() == (2 if dt == "f32" else 1)
    check(q.cpu(), k.cpu(), v.cpu(), cu, True, o, lse, tensor_cores=dt != "f32")
    assert big[:, :H].eq(3.0).all()
    # heads outermost (the dense layout), and rows that are not 16-byte aligned
    qh, kh, vh = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    o2, _ = api.attention_packed(qh, kh, vh, cu.cuda(), is_causal=True, return_lse=True)
    assert torch.equal(o2, o)
    pad = torch.zeros(T, H + 2 * Hkv, D + 1, dtype=DT[dt], device="cuda")
    pad[..., 1:] = x
    y = pad[..., 1:]
    o3, l3 = api.attention_packed(y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:], cu.cuda(),
                                  is_causal=True, return_lse=True)
    assert api.last_path() == 2
    check(q.cpu(), k.cpu(), v.cpu(), cu, True, o3, l3, tensor_cores=False)
    # one key/value row for all tokens (a broadcast)
    o4, l4 = api.attention_packed(q, k[:1].expand(T, Hkv, D), v, cu.cuda(), return_lse=True)
    check(q.cpu(), k[:1].expand(T, Hkv, D).cpu(), v.cpu(), cu, False, o4, l4, tensor_cores=False)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_bad_offsets_are_skipped_and_reported(dt, causal):
    q, k, v, cu = make([50, 60, 40], 4, 2, 64, dt, seed=7)
    good, _ = run(q, k, v, cu, causal)
    for bad in ([0, 50, 40, 40], [0, 50, 110, 151], [-1, 50, 110, 150]):
        out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
        run(q, k, v, torch.tensor(bad, dtype=torch.int32), causal, out=out)
        assert api.device_status() == _abi.JVP_ERR_INDEX
        for b in range(3):
            r0, r1 = bad[b], bad[b + 1]
            if 0 <= r0 <= r1 <= 150 and [r0, r1] == cu[b:b + 2].tolist():
                assert torch.equal(out[r0:r1], good[r0:r1])
        if bad[3] == 151:
            assert out[110:].eq(5.0).all()
        if bad[0] == -1:
            assert out[:50].eq(5.0).all()


def test_many_offsets_are_checked():
    q, k, v, cu = make([2] * 100, 2, 2, 64, "bf16", seed=7)
    cu[70] = 300
    run(q, k, v, cu, True)
    assert api.device_status() == _abi.JVP_ERR_INDEX


def test_matches_the_dense_attention_on_equal_lengths():
    B, H, Hkv, N, D = 3, 8, 2, 300, 128
    q, k, v, cu = make([N] * B, H, Hkv, D, "bf16", seed=9)
    o, lse = run(q, k, v, cu, True)
    dense = [t.view(B, N, -1, D).transpose(1, 2).cuda() for t in (q, k, v)]
    od, ld = api.attention(*dense, is_causal=True, return_lse=True)
    check(q, k, v, cu, True, od.transpose(1, 2).reshape(o.shape),
          ld.permute(1, 0, 2).reshape(lse.shape))
    check(q, k, v, cu, True, o, lse)


def test_empty_problems():
    z = torch.zeros(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    o, lse = api.attention_packed(z, z, z, torch.zeros(3, dtype=torch.int32, device="cuda"),
                                  return_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    x = torch.ones(5, 4, 64, device="cuda", dtype=torch.bfloat16)
    out = torch.full_like(x, 2.0)
    for cu in ([0], [2, 2, 2], [5, 5]):
        api.attention_packed(x, x, x, torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out)
    assert out.eq(2.0).all()


def test_another_stream_and_a_graph_that_follows_the_offsets():
    q, k, v, cu = make([300, 100, 50], 4, 1, 128, "bf16", seed=10)
    dq, dk, dv, dcu = (t.cuda() for t in (q, k, v, cu))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = api.attention_packed(dq, dk, dv, dcu, is_causal=True, return_lse=True)
    torch.cuda.current_stream().wait_stream(s)
    check(q, k, v, cu, True, o, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = api.attention_packed(dq, dk, dv, dcu, is_causal=True, return_lse=True)
    for lens in ([300, 100, 50], [1, 448, 1], [0, 20, 430]):
        new = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
        dcu.copy_(new)
        graph.replay()
        check(q, k, v, new, True, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_prompt_and_the_tokens_after_it(e4m3):
    """As a server runs them: packed prompts, their rows into the cache, then a
    token at a time; each token's output is the last row of attention over
    everything so far."""
    H, Hkv, D, page, lens, steps = 8, 2, 64, 16, [37, 5, 64], 3
    B, most = len(lens), 6
    q, k, v, cu = make([n + steps for n in lens], H, Hkv, D, "bf16", seed=11)
    rows = [torch.arange(int(cu[b]), int(cu[b]) + lens[b]) for b in range(B)]
    first = torch.cat(rows)
    pcu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc = torch.zeros(B * most, Hkv, page, D, device="cuda").to(dt)
    vc = torch.zeros_like(kc)
    ks, vs = ([torch.zeros(kc.shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)]
              if e4m3 else (None, None))
    table = torch.randperm(B * most, generator=torch.Generator().manual_seed(1)).int().view(B, most).cuda()
    args = dict(k_scale=ks, v_scale=vs)
    pq, pk, pv = (t[first].cuda() for t in (q, k, v))
    o, lse = api.attention_packed(pq, pk, pv, pcu.cuda(), is_causal=True, return_lse=True)
    check(pq.cpu(), pk.cpu(), pv.cpu(), pcu, True, o, lse)
    api.cache_write(pk, pv, kc, vc, table, None, pcu.cuda(), **args)
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for t in range(steps):
        at = torch.tensor([int(cu[b]) + lens[b] + t for b in range(B)])
        api.cache_write(k[at].cuda(), v[at].cuda(), kc, vc, table, lens_d, **args)
        lens_d += 1
        o, lse = api.attention_decode(q[at].cuda(), kc, vc, table, lens_d, return_lse=True, **args)
        for b in range(B):
            n = lens[b] + t + 1
            r = slice(int(cu[b]), int(cu[b]) + n)
            rk, rv = k[r], v[r]
            if e4m3:
                rk, rv = api.cache_read(kc, vc, table[b:b + 1], None,
                                        torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                        num_rows=n, dtype=torch.float32, **args)
                # half a step of e4m3 (2^-4) of the value or of its smallest step
                top = k[r].float().abs().amax(-1, keepdim=True)
                assert (rk.cpu() - k[r].float()).abs().le(
                    2.0 ** -4 * k[r].float().abs() + top * 2.0 ** -17).all()
            for h in range(H):
                ref = attend(f64(q[at[b], h])[None], f64(rk[:, h // 4]), f64(rv[:, h // 4]),
                             np.ones((1, n), bool), D ** -0.5)
                b_o, b_lse = bounds(*ref, n, D, 2.0 ** -8, 2.0 ** -8, True)
                assert (np.abs(f64(o[b, h]) - ref[0][0]) <= b_o[0]).all()
                assert abs(f64(lse[b, h]) - ref[1][0]) <= b_lse[0]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [2, 40])  # (few heads: one query tile per CTA at D = 128)
@pytest.mark.parametrize("n", [100, 300, 1000, 1290, 1700])
def test_a_query_tile_on_its_own_keeps_its_running_maximum(n, H, D, causal):
    """Lengths whose last work item has one query tile only (its steps run
    through the score buffers alone), with keys that grow so that most tiles
    rescale; and many such items side by side."""
    q, k, v, cu = make([n, 128 * 5 + 1, n], H, H, D, "bf16", seed=n)
    ramp = torch.cat([torch.linspace(0.2, 8.0, int(m)) for m in (cu[1:] - cu[:-1])])[:, None, None]
    q, k = (q.abs() * 2).bfloat16(), (k.abs() * ramp).bfloat16()
    o, lse = run(q, k, v, cu, causal)
    check(q, k, v, cu, causal, o, lse, heads=[0, H - 1])
    for _ in range(5):
        o2, lse2 = run(q, k, v, cu, causal)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,Hkv,D", [(7, 1, 64), (3, 1, 64), (7, 1, 128), (8, 8, 64), (16, 2, 128)])
def test_many_calls_give_the_same_bits(H, Hkv, D):
    """Two tiles per CTA run at their own pace (one may be masked more than the
    other): no order of theirs may show."""
    q, k, v, cu = (t.cuda() for t in make(LONG, H, Hkv, D, "bf16", seed=1))
    o, lse = api.attention_packed(q, k, v, cu, is_causal=True, return_lse=True)
    for _ in range(60):
        o2, lse2 = api.attention_packed(q, k, v, cu, is_causal=True, return_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
