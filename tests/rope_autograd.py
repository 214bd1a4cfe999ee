"""Derivatives of autograd.norm_rope in the ways that torch offers them.

Each way takes a function f(q, k, wq, wk) -> (q, k), its arguments, their tangents
and cotangents, and returns tensors; the same way applied to the float64 definition
says what they should be.  `plain_kernels` stands in for the kernels without a GPU: what
they compute, on plain tensors only, with no history and no tangents.
"""

import itertools

import rope_ref
import torch
import torch.autograd.forward_ad as fwAD
from forward_mode_flash_gb300 import api, autograd

EPS = 1e-5
B, H, HKV, N, D = 2, 4, 2, 5, 16


# ---------------------------------------------------------------- stand-ins
def _raw(t):
    if t is None:
        return None
    if torch._C._functorch.is_functorch_wrapped_tensor(t):
        raise RuntimeError("a tensor without storage")
    assert t.stride(-1) == 1
    return t.detach()


def _kernel(f):
    def call(*args):
        with torch.no_grad(), fwAD._set_fwd_grad_enabled(False):
            return f(*(_raw(t) if isinstance(t, torch.Tensor) else t for t in args))
    return call


def _side(x, t, gy, gt, w, table, eps, interleaved):
    """Values, tangents and gradients of one side by their formulas, in float64."""
    x, t, gy, gt, w, table = (None if z is None else z.double() for z in (x, t, gy, gt, w, table))
    mean = lambda z: z.mean(-1, keepdim=True)  # noqa: E731
    turn = lambda z: rope_ref.rotate(z, table, interleaved)  # noqa: E731
    half = table.shape[-1] // 2
    other_way = torch.cat((table[..., :half], -table[..., half:]), -1)
    r = (mean(x * x) + eps).rsqrt()
    n = r * x
    out = {"y": turn(w * n)}
    a = rope_ref.rotate(gy, other_way, interleaved)
    u = w * a
    out["gx"], gw = r * (u - n * mean(u * n)), a * n
    if t is not None:
        m = mean(n * t)
        dn = r * (t - m * n)
        out["dy"] = turn(w * dn)
        b = rope_ref.rotate(gt, other_way, interleaved)
        v = w * b
        out["gdx"] = r * (v - n * mean(v * n))
        out["gx"] = out["gx"] + r * r * (n * (3 * m * mean(v * n) - mean(v * t)) - t * mean(v * n) - m * v)
        gw = gw + b * dn
    out["gw"] = gw.sum((0, 1, 2))
    return out


def _sides(tensors, g, table, positions, weights, eps, interleaved):
    assert positions is None
    g = g or [torch.zeros_like(z) for z in tensors[:2]] * 2
    return [_side(tensors[i], tensors[2 + i], g[i], g[2 + i], weights[i], table, eps, interleaved)
            for i in (0, 1)]


def plain_kernels(monkeypatch):
    def rows(q, k, dq, dk, table, positions, wq, wk, eps, il):
        s = _sides((q, k, dq, dk), None, table, positions, (wq, wk), eps, il)
        return tuple(x[n].to(q.dtype) for n in (("y",) if dq is None else ("y", "dy")) for x in s)

    def grads(tensors, g, table, positions, wq, wk, eps, il):
        s = _sides(tensors, g, table, positions, (wq, wk), eps, il)
        names = ("gx",) if tensors[2] is None else ("gx", "gdx")
        return (*(x[n].to(tensors[0].dtype) for n in names for x in s),
                *(x["gw"].float() for x in s))

    monkeypatch.setattr(api, "norm_rope", _kernel(
        lambda q, k, *rest: rows(q, k, None, None, *rest)))
    monkeypatch.setattr(api, "norm_rope_dual", _kernel(rows))
    monkeypatch.setattr(api, "norm_rope_bwd", _kernel(
        lambda q, k, a, b, *rest: grads((q, k, None, None), (a, b, None, None), *rest)))
    monkeypatch.setattr(api, "norm_rope_bwd_dual", _kernel(
        lambda q, k, dq, dk, a, b, c, d, *rest: grads((q, k, dq, dk), (a, b, c, d), *rest)))


# ---------------------------------------------------------------- data
NAMES = ("q", "k", "wq", "wk")
SOME = [s for n in (1, 2, 3, 4) for s in itertools.combinations(range(4), n)]


def data(dtype=torch.float32, seed=0):
    """(arguments, their tangents, two pairs of cotangents of the results)."""
    g = torch.Generator().manual_seed(seed)
    shapes = ((B, H, N, D), (B, HKV, N, D), (D,), (D,))
    r = lambda s: torch.randn(s, generator=g).to(dtype)  # noqa: E731
    args = [r(s) for s in shapes[:2]] + [(1 + 0.2 * r(s)).to(dtype) for s in shapes[2:]]
    return args, [r(s) for s in shapes], [r(s) for s in shapes[:2] * 2]


def own(table):
    return lambda q, k, wq, wk: autograd.norm_rope(q, k, table, None, wq, wk, EPS)


def plain(table):
    return lambda q, k, wq, wk: tuple(rope_ref.norm_rope(x, w, table.double(), EPS, False)
                                      for x, w in ((q, wq), (k, wk)))


def loss(y, t, c):
    return sum((a * b).sum() for a, b in zip((*y, *t), c))


def at(f, args, which):
    """f of the arguments `which`, the others as they are."""
    def g(*some):
        full = list(args)
        for i, x in zip(which, some):
            full[i] = x
        return f(*full)
    return g


# ---------------------------------------------------------------- ways
def train_through_jvp(f, args, tangents, c, which):
    """Values, tangents for tangents of some arguments, and gradients of both by all."""
    leaves = [x.clone().requires_grad_() for x in args]
    moving = [tangents[i].clone().requires_grad_() for i in which]
    y, t = torch.func.jvp(at(f, leaves, which), tuple(leaves[i] for i in which), tuple(moving))
    return (*y, *t, *torch.autograd.grad(loss(y, t, c), leaves + moving))


def train_through_dual_tensors(f, args, tangents, c, which):
    """The same by torch.autograd.forward_ad, gradients taken behind its level."""
    leaves = [x.clone().requires_grad_() for x in args]
    moving = [tangents[i].clone().requires_grad_() for i in which]
    with fwAD.dual_level():
        full = list(leaves)
        for i, x in zip(which, moving):
            full[i] = fwAD.make_dual(leaves[i], x)
        pairs = [fwAD.unpack_dual(x) for x in f(*full)]
    y, t = [p.primal for p in pairs], [p.tangent for p in pairs]
    assert any(x is not None for x in t)
    t = [torch.zeros_like(a) if b is None else b for a, b in zip(y, t)]  # (of a side without)
    return (*y, *t, *torch.autograd.grad(loss(y, t, c), leaves + moving))


def values_by_dual_tensors(f, args, tangents, c, which):
    """Without the gradients: those of values and tangents come from two calls there, and
    autograd adds what each has rounded, as for any tensor with two uses."""
    return train_through_dual_tensors(f, args, tangents, c, which)[:4]


def grad_of_jvp(f, args, tangents, c, which):
    """torch.func.grad by all arguments of a loss of values and tangents for some."""
    def of(*args):
        return loss(*torch.func.jvp(at(f, args, which), tuple(args[i] for i in which),
                                    tuple(tangents[i] for i in which)), c)
    return torch.func.grad(of, argnums=(0, 1, 2, 3))(*args)


def grad_of_others(f, args, tangents, c, which):
    """The same by the arguments without tangents alone."""
    rest = tuple(i for i in range(4) if i not in which)

    def of(*some):
        return loss(*torch.func.jvp(at(at_list(f, args, rest, some), args, which),
                                    tuple(args[i] for i in which),
                                    tuple(tangents[i] for i in which)), c)
    return torch.func.grad(of, argnums=tuple(range(len(rest))))(*(args[i] for i in rest))


def at_list(f, args, which, some):
    """f with the arguments `which` replaced by some, whatever it is given there."""
    def g(*full):
        full = list(full)
        for i, x in zip(which, some):
            full[i] = x
        return f(*full)
    return g


def gradients(f, args, tangents, c, which):
    """torch.func.grad of a loss of the values."""
    return torch.func.grad(lambda *x: loss(f(*x), (), c), argnums=which)(*args)


def pulled_back(f, args, tangents, c, which):
    """torch.func.vjp by some arguments."""
    y, back = torch.func.vjp(at(f, args, which), *(args[i] for i in which))
    return (*y, *back(tuple(c[:2])))


def tangents_of_gradients(f, args, tangents, c, which):
    """torch.func.jvp over torch.func.grad, of a loss whose cotangents depend on the values."""
    def grads(*some):
        return torch.func.grad(lambda *x: sum((a * b).sin().sum() for a, b in zip(f(*x), c)),
                               argnums=(0, 1, 2, 3))(*at_list(lambda *x: x, args, which, some)(*args))
    g, t = torch.func.jvp(grads, tuple(args[i] for i in which), tuple(tangents[i] for i in which))
    return (*g, *t)


def tangents_of_gradients_by_dual_tensors(f, args, tangents, c, which):
    """The same by torch.autograd.forward_ad and torch.autograd.grad within its level."""
    with fwAD.dual_level():
        leaves = [x.clone().requires_grad_() for x in args]
        full = list(leaves)
        for i in which:
            full[i] = fwAD.make_dual(leaves[i], tangents[i])
        g = torch.autograd.grad(sum((a * b).sin().sum() for a, b in zip(f(*full), c)), leaves)
        pairs = [fwAD.unpack_dual(x) for x in g]
        return [p.primal.clone() for p in pairs] + [
            torch.zeros_like(p.primal) if p.tangent is None else p.tangent.clone() for p in pairs]


def compare(way, to, table, *rest, dtype=torch.float32, **kw):
    """Asserts that a way gives the same of the framework's function and of the definition's."""
    args, tangents, c = data(dtype)
    got = way(own(to(table)), *([to(x) for x in z] for z in (args, tangents, c)), *rest, **kw)
    want = way(plain(table), *([x.double() for x in z] for z in (args, tangents, c)), *rest, **kw)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        # some three hundred roundings of 2^-24: a row's sums have 16 terms, the weights'
        # gradients 40 rows; and one of the result's type
        step = torch.finfo(a.dtype).eps / 2 if a.dtype != torch.float32 else 0.0
        a = a.detach().double().cpu()
        bound = step * b.abs() + (1 + step) * 2e-5 * max(1.0, b.abs().max())
        assert ((a - b).abs() <= bound).all(), ((a - b).abs() / bound).max()
