"""Norms and rotation of dense queries and keys, their tangents and gradients,
against float64 (bounds derived in rope_ref.py)."""

import pytest
import torch

import rope_ref
from forward_mode_flash_gb300 import _abi, api, autograd, build

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(autouse=True)
def _status_clear():
    api.device_status()
    yield
    assert api.device_status() == _abi.JVP_OK


def make(B, H, Hkv, N, D, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    rows = [torch.randn(B, h, N, D, generator=g).to(DT[dt]) for _ in range(4) for h in (H, Hkv)]
    w = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)]
    return rows, w


def run(rows, w, table, positions=None, tangents=True, interleaved=False, eps=EPS):
    """Outputs and gradients on the GPU, by side."""
    c = lambda z: None if z is None else z.cuda()  # noqa: E731
    q, k, dq, dk, gq, gk, gdq, gdk = (c(z) for z in rows)
    kw = dict(rope=c(table), positions=c(positions), q_weight=c(w[0]), k_weight=c(w[1]), eps=eps,
              interleaved=interleaved)
    if tangents:
        y = api.norm_rope_dual(q, k, dq, dk, **kw)
        g = api.norm_rope_bwd_dual(q, k, dq, dk, gq, gk, gdq, gdk, **kw)
        return [{"y": y[i], "dy": y[2 + i], "gx": g[i], "gdx": g[2 + i], "gw": g[4 + i]}
                for i in (0, 1)]
    y = api.norm_rope(q, k, **kw)
    g = api.norm_rope_bwd(q, k, gq, gk, **kw)
    return [{"y": y[i], "gx": g[i], "gw": g[2 + i]} for i in (0, 1)]


def check(got, rows, w, table, positions=None, tangents=True, interleaved=False, eps=EPS):
    N = rows[0].shape[2]
    at = None
    if table is not None:
        at = table[:N] if positions is None else table[positions.long()]
        at = at[:, None] if at.dim() == 3 else at
    for i in (0, 1):
        x, t, gy, gt = rows[i], rows[2 + i], rows[4 + i], rows[6 + i]
        rope_ref.check_side(got[i], x, t if tangents else None, gy, gt if tangents else None, w[i],
                            at, eps, interleaved)


SHAPES = [  # B, H, Hkv, N, D, rotated columns
    (2, 4, 2, 37, 128, 128), (1, 3, 1, 5, 64, 64), (2, 2, 2, 33, 128, 64), (1, 16, 4, 1, 128, 128),
    (3, 2, 1, 19, 96, 96), (1, 6, 2, 50, 80, 48), (2, 3, 3, 9, 40, 40), (1, 2, 1, 7, 40, 32),
    (1, 2, 2, 11, 33, 20), (2, 1, 1, 3, 2, 2), (1, 1, 1, 6, 8, 8), (1, 2, 1, 700, 16, 16),
    (1, 5, 0, 4, 64, 64), (1, 0, 5, 4, 64, 64)]


@pytest.mark.parametrize("tangents", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norms_and_rotation(shape, dt, interleaved, tangents):
    *sizes, rot = shape
    rows, w = make(*sizes, dt, seed=rot)
    table = api.rope_table(sizes[3] + 3, rot)
    got = run(rows, w, table, None, tangents, interleaved)
    check(got, rows, w, table, None, tangents, interleaved)


@pytest.mark.parametrize("tangents", [False, True])
@pytest.mark.parametrize("dt,D", [("f32", 64), ("bf16", 128), ("f16", 50)])
def test_rotation_alone_and_norms_alone(dt, D, tangents):
    rows, w = make(2, 4, 1, 21, D, dt)
    table = api.rope_table(21, D)
    check(run(rows, [None, None], table, None, tangents), rows, [None, None], table, None, tangents)
    check(run(rows, w, None, None, tangents), rows, w, None, None, tangents)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shared", [False, True])
def test_positions(dt, shared):
    """Positions in any order, twice the same, far ones; one row for all sequences or one each."""
    rows, w = make(3, 2, 1, 40, 64, dt)
    table = api.rope_table(5000, 64)
    g = torch.Generator().manual_seed(1)
    positions = torch.randint(0, 5000, (40,) if shared else (3, 40), generator=g).int()
    positions[..., 3] = positions[..., 4]
    positions[..., 5] = 4999
    check(run(rows, w, table, positions), rows, w, table, positions)


@pytest.mark.parametrize("wdt", [torch.float16, torch.bfloat16])
def test_weights_of_16_bits(wdt):
    rows, w = make(2, 2, 2, 9, 128, "bf16")
    w = [x.to(wdt) for x in w]
    table = api.rope_table(9, 128)
    check(run(rows, w, table), rows, w, table)


@pytest.mark.parametrize("dt,D", [("f32", 64), ("bf16", 128)])
def test_strides(dt, D):
    """Rows as a projection leaves them ([B, N, heads, D] seen as [B, heads, N, D]), rows off
    their alignment, and cotangents shared by the heads."""
    rows, w = make(2, 4, 4, 19, D, dt)
    table = api.rope_table(19, D)
    want = run(rows, w, table)
    t = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in rows]
    for a, b in zip(want, run(t, w, table)):
        assert all(torch.equal(a[n], b[n]) for n in a)
    c = [x.cuda() for x in rows]
    odd = []
    for x in c:
        wide = torch.zeros(*x.shape[:3], D + 1, dtype=x.dtype, device="cuda")
        odd.append(wide[..., 1:])
        odd[-1].copy_(x)
    kw = dict(rope=table.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda(), eps=EPS)
    y, g = api.norm_rope_dual(*odd[:4], **kw), api.norm_rope_bwd_dual(*odd, **kw)
    check([{"y": y[i], "dy": y[2 + i], "gx": g[i], "gdx": g[2 + i], "gw": g[4 + i]} for i in (0, 1)],
          rows, w, table)
    shared = [x[:, :1].expand(-1, 4, -1, -1) for x in c[4:]]
    g = api.norm_rope_bwd_dual(*c[:4], *shared, **kw)
    check([{"gx": g[i], "gdx": g[2 + i], "gw": g[4 + i]} for i in (0, 1)],
          rows[:4] + [x[:, :1].expand(-1, 4, -1, -1) for x in rows[4:]], w, table)


@pytest.mark.parametrize("dt,D", [("f32", 64), ("bf16", 128), ("f16", 30)])
def test_many_rows(dt, D):
    """More rows than the GPU has warps at once; the same bits twice."""
    rows, w = make(2, 8, 2, 3000, D, dt)
    table = api.rope_table(3000, D)
    got = run(rows, w, table)
    check(got, rows, w, table)
    for a, b in zip(got, run(rows, w, table)):
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_of_zeros_and_large_rows(dt):
    """A row of zeros is normalised to zeros (eps), large and small ones to the same size."""
    rows, w = make(1, 3, 3, 8, 64, dt)
    for x in rows[:2]:
        x[0, :, 0] = 0
        x[0, :, 1] *= 2.0 ** 40
        x[0, :, 2] *= 2.0 ** -20
    table = api.rope_table(8, 64)
    check(run(rows, w, table), rows, w, table)


def test_no_rows():
    rows, w = make(2, 3, 1, 0, 64, "bf16")
    got = run(rows, w, api.rope_table(4, 64))
    assert got[0]["y"].shape == (2, 3, 0, 64) and (got[0]["gw"] == 0).all()
    assert (got[1]["gw"] == 0).all()


@pytest.mark.parametrize("D", [64, 30])
def test_positions_out_of_range_are_reported(D):
    rows, w = make(1, 2, 1, 6, D, "bf16")
    table = api.rope_table(10, D)
    positions = torch.tensor([[0, 9, 10, -1, 4, 2147483647]], dtype=torch.int32)
    got = run(rows, w, table, positions, eps=0.0)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    keep = torch.tensor([0, 1, 4])
    kept = [x[:, :, keep] for x in rows]
    for side in got:
        for n in side:
            if n != "gw":
                side[n] = side[n][:, :, keep.cuda()]
    check(got, kept, w, table, positions[:, keep], eps=0.0)


# ---------------------------------------------------------------- autograd
def reference(q, k, w, table, eps=EPS):
    return [rope_ref.norm_rope(x, y, table, eps, False) for x, y in zip((q, k), w)]


def test_gradients_by_autograd():
    rows, w = make(2, 4, 2, 21, 64, "f32")
    table = api.rope_table(21, 64)
    leaves = [x.cuda().requires_grad_() for x in (*rows[:2], *w)]
    y = autograd.norm_rope(*leaves[:2], table.cuda(), None, *leaves[2:], EPS)
    g = torch.autograd.grad(y, leaves, [x.cuda() for x in rows[4:6]])
    check([{"y": y[i].detach(), "gx": g[i], "gw": g[2 + i]} for i in (0, 1)], rows, w, table,
          tangents=False)
    # only one output in the loss, and weights of 16 bits
    leaves = [x.cuda().requires_grad_() for x in (*rows[:2], *(x.bfloat16() for x in w))]
    q, _ = autograd.norm_rope(*leaves[:2], table.cuda(), None, *leaves[2:], EPS)
    g = torch.autograd.grad(q.sum(), leaves)
    assert (g[1] == 0).all() and (g[3] == 0).all() and g[2].dtype == torch.bfloat16


def test_gradients_against_differences():
    """Fourth-order differences of the float32 kernel along random directions: the
    truncation is h^4 / 30 of a fifth derivative (a few units), the rounding of the
    values 2^-22 / h of their norm."""
    rows, w = make(1, 2, 2, 5, 32, "f32", seed=4)
    table = api.rope_table(5, 32).cuda()
    x = [z.cuda() for z in (*rows[:2], *w)]
    c = [z.cuda() for z in rows[4:6]]
    v = [torch.randn(z.shape, generator=torch.Generator().manual_seed(7)).cuda() for z in x]

    def loss(h):
        y = api.norm_rope(*(a + h * b for a, b in zip(x[:2], v)), table, None,
                          *(a + h * b for a, b in zip(x[2:], v[2:])), EPS)
        return sum((a.double() * b.double()).sum() for a, b in zip(y, c))

    h = 0.02
    slope = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
    g = api.norm_rope_bwd(*x[:2], *c, table, None, *x[2:], EPS)
    want = sum((a.double() * b.double()).sum() for a, b in zip(g, v))
    size = sum(a.double().norm() * b.double().norm() for a, b in zip(g, v))
    assert abs(slope - want) <= 1e-3 * size


@pytest.mark.parametrize("weights", [False, True])
def test_training_through_a_jvp(weights):
    """torch.func.jvp of norms, rotation and attention, and gradients of both of its
    results, against the same model in float64 without the framework."""
    g = torch.Generator().manual_seed(2)
    B, H, Hkv, N, D = 1, 4, 2, 24, 32
    q, dq, c, ct = (torch.randn(B, H, N, D, generator=g) for _ in range(4))
    k, dk, v, dv = (torch.randn(B, Hkv, N, D, generator=g) for _ in range(4))
    w = [1 + 0.2 * torch.randn(D, generator=g) for _ in range(2)]
    dw = [0.3 * torch.randn(D, generator=g) for _ in range(2)]
    table = api.rope_table(N, D)

    def plain(q, k, v, wq, wk):
        a, b = reference(q, k, (wq, wk), table.double())
        b, v = (x.repeat_interleave(H // Hkv, 1) for x in (b, v))
        s = (a @ b.transpose(-1, -2) / D ** 0.5).masked_fill(
            torch.ones(N, N, dtype=torch.bool).triu(1), float("-inf"))
        return s.softmax(-1) @ v

    def own(q, k, v, wq, wk):
        a, b = autograd.norm_rope(q, k, table.cuda(), None, wq, wk, EPS)
        return autograd.jvp_attention(a, b, v, is_causal=True)

    def both(f, to):
        leaves = [to(x).requires_grad_() for x in (q, k, v, *w)]
        t = [to(x) for x in (dq, dk, dv)]
        if weights:
            o, to_ = torch.func.jvp(f, tuple(leaves), (*t, *(to(x) for x in dw)))
        else:
            o, to_ = torch.func.jvp(lambda a, b, d: f(a, b, d, *leaves[3:]), tuple(leaves[:3]),
                                    tuple(t))
        grads = torch.autograd.grad((o * to(c)).sum() + (to_ * to(ct)).sum(), leaves)
        return [x.detach().double().cpu() for x in (o, to_, *grads)]

    # fp32 throughout: some hundred roundings of 2^-24 on values of up to a few units
    for a, b in zip(both(own, lambda x: x.cuda()), both(plain, lambda x: x.double())):
        assert (a - b).abs().max() <= 2e-5 * max(1.0, b.abs().max())


def test_forward_mode_without_torch_func():
    rows, w = make(1, 2, 1, 6, 64, "f32")
    table = api.rope_table(6, 64)
    q, k, dq, dk = (x.cuda() for x in rows[:4])
    w = [x.cuda() for x in w]
    want = api.norm_rope_dual(q, k, dq, dk, table.cuda(), None, *w, EPS)
    import torch.autograd.forward_ad as fwAD
    with fwAD.dual_level():
        y = autograd.norm_rope(fwAD.make_dual(q, dq), fwAD.make_dual(k, dk), table.cuda(), None, *w,
                               EPS)
        got = [fwAD.unpack_dual(x) for x in y]
    assert all(torch.equal(got[i][0], want[i]) and torch.equal(got[i][1], want[2 + i])
               for i in (0, 1))


def test_captured_graph_follows_its_inputs():
    rows, w = make(2, 4, 2, 50, 128, "bf16")
    table = api.rope_table(50, 128).cuda()
    x = [z.cuda() for z in rows]
    kw = dict(rope=table, q_weight=w[0].cuda(), k_weight=w[1].cuda(), eps=EPS)
    api.norm_rope_bwd_dual(*x, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = api.norm_rope_dual(*x[:4], **kw), api.norm_rope_bwd_dual(*x, **kw)
    for z in x:
        z.mul_(0.5).add_(0.25)
    graph.replay()
    for a, b in zip((*y, *g), (*api.norm_rope_dual(*x[:4], **kw), *api.norm_rope_bwd_dual(*x, **kw))):
        assert torch.equal(a, b)


def test_another_stream():
    rows, w = make(2, 4, 2, 500, 128, "bf16")
    table = api.rope_table(500, 128).cuda()
    x = [z.cuda() for z in rows]
    kw = dict(rope=table, q_weight=w[0].cuda(), k_weight=w[1].cuda(), eps=EPS)
    want = api.norm_rope_bwd_dual(*x, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(api.norm_rope_bwd_dual(*x, **kw))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_a_captured_training_step():
    """Values and gradients captured together; replays follow the inputs, and eager graphs of the
    same leaves come before and after."""
    rows, w = make(1, 4, 2, 40, 64, "bf16")
    table = api.rope_table(40, 64).cuda()
    leaves = [x.cuda().requires_grad_() for x in (*rows[:2], *w)]
    c = [x.cuda() for x in rows[4:6]]

    def step():
        y = autograd.norm_rope(*leaves[:2], table, None, *leaves[2:], EPS)
        return torch.autograd.grad(y, leaves, c)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        with torch.no_grad():
            for x in (*leaves, *c):
                x.mul_(0.75).add_(0.125)
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_gradients_of_gradients_are_refused():
    rows, w = make(1, 2, 1, 6, 32, "f32")
    leaves = [x.cuda().requires_grad_() for x in (*rows[:2], *w)]
    y = autograd.norm_rope(*leaves[:2], api.rope_table(6, 32).cuda(), None, *leaves[2:], EPS)
    g = torch.autograd.grad((y[0] ** 2).sum(), leaves[0], create_graph=True)[0]
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


@pytest.mark.parametrize("tangents", [False, True])
@pytest.mark.parametrize("dt,D,rot", [("bf16", 64, 64), ("f32", 33, 6)])
def test_rotations_alone_do_not_read_the_rows_backwards(dt, D, rot, tangents):
    """The C entry takes NULL for them."""
    rows, _ = make(2, 3, 1, 9, D, dt)
    q, k, dq, dk, *c = (x.cuda() for x in rows)
    table = api.rope_table(9, rot).cuda()
    if tangents:
        want = api.norm_rope_bwd_dual(q, k, dq, dk, *c, table)[:4]
    else:
        want, c = api.norm_rope_bwd(q, k, *c[:2], table)[:2], c[:2]
    out = [torch.full_like(x, 7.0) for x in want]
    st = [_abi.Strides(*x.stride()[:3], 1) for x in (q, k) * 4]
    p = lambda t, i: t[i].data_ptr() if i < len(t) else None  # noqa: E731
    lib = _abi.load()
    rope = _abi.Rope(table.data_ptr(), 9, rot, 0, 0, None, None, 0.0)
    torch.cuda.synchronize()
    r = lib.jvp_attn_norm_rope_bwd(
        _abi.Shape(2, 3, 9, 9, D, 1), {"bf16": _abi.JVP_BF16, "f32": _abi.JVP_F32}[dt], rope, None, 0,
        None, None, None, None, *(p(c, i) for i in range(4)), (_abi.Strides * 8)(*st),
        *(p(out, i) for i in range(4)), (_abi.Strides * 4)(*st[:4]), None, None, None, 0, None)
    assert r == _abi.JVP_OK
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_broadcast_inputs():
    """Queries and keys expanded over the batch: the gradients of what was expanded are sums."""
    rows, w = make(1, 4, 2, 30, 64, "f32", seed=8)
    table = api.rope_table(30, 64).cuda()
    c = [torch.randn(3, h, 30, 64, generator=torch.Generator().manual_seed(h)).cuda() for h in (4, 2)]
    got = []
    for expand in (lambda x: x.expand(3, -1, -1, -1), lambda x: x.repeat(3, 1, 1, 1)):
        leaves = [x.cuda().requires_grad_() for x in (*rows[:2], *w)]
        y = autograd.norm_rope(*(expand(x) for x in leaves[:2]), table, None, *leaves[2:], EPS)
        got.append((*y, *torch.autograd.grad(y, leaves, c)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
