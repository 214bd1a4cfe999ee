"""Norms of queries and keys and their rotation in float64, with error bounds.

norm_rope(x, w, table rows) is written with complex numbers; tangents and
gradients come from automatic differentiation of it.

Bounds (s = 2^-24, one rounding of fp32): a row's sum of squares has D products
and sums, then the division, eps, the reciprocal root (2 units in the last place)
and three products: r is off by (D / 2 + 8) s relatively (the root halves the
sum's share).  A product of the row with r, w, cos or sin, and a sum of two, add
one s each.  Everything after that is a sum of terms, so errors are bounded by
the same formula over magnitudes: `norm_rope_bounds` evaluates it with absolute
values.  On top one rounding of the result's type.
"""

import torch

S = 2.0 ** -24


def rotate(x, table, interleaved):
    """x [.., D] by rows [.., dim] of cosines and sines."""
    if table is None:
        return x
    half = table.shape[-1] // 2
    unit = torch.complex(table[..., :half], table[..., half:])
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    else:
        a, b = x[..., :half], x[..., half:2 * half]
    y = torch.complex(a, b) * unit
    if interleaved:
        y = torch.stack((y.real, y.imag), -1).flatten(-2)
    else:
        y = torch.cat((y.real, y.imag), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def norm_rope(x, w, table, eps, interleaved):
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    return rotate(x, table, interleaved)


def _rotate_abs(x, table, interleaved):
    """Bound of the magnitudes a rotation sums: |a cos| + |b sin|, |a sin| + |b cos|."""
    if table is None:
        return x
    half = table.shape[-1] // 2
    c, s = table[..., :half].abs(), table[..., half:].abs()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * c + b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * c + b * s, a * s + b * c), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def magnitudes(x, t, gy, gt, w, table, eps, interleaved):
    """Sums of the magnitudes of the terms of every output (y, dy, gx, gdx, gw)."""
    D = x.shape[-1]
    r = 1.0 if w is None else (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = r * x.abs()
    wa = 1.0 if w is None else w.abs()
    mean = lambda z: z.mean(-1, keepdim=True)  # noqa: E731
    out = {"y": _rotate_abs(wa * n, table, interleaved)}
    a = _rotate_abs(gy.abs(), table, interleaved)
    u = wa * a
    out["gx"] = u if w is None else r * (u + n * mean(u * n))
    gw = a * n
    if t is not None:
        ta = t.abs()
        m = mean(n * ta)
        dn = ta if w is None else r * (ta + n * m)
        out["dy"] = _rotate_abs(wa * dn, table, interleaved)
        b = _rotate_abs(gt.abs(), table, interleaved)
        v = wa * b
        if w is None:
            out["gdx"] = v
        else:
            p, q = mean(v * ta), mean(v * n)
            out["gdx"] = r * (v + n * q)
            out["gx"] = out["gx"] + r * r * (n * (3 * m * q + p) + ta * q + m * v)
            gw = gw + b * dn
    if w is not None:
        out["gw"] = gw.sum(tuple(range(gw.dim() - 1)))
        out["rows"] = gw.numel() // D
    return out


def side_64(x, t, gy, gt, w, table, eps, interleaved):
    """Float64 outputs of one side: y, dy, gx, gdx, gw (None where there is none)."""
    x, t, gy, gt = (None if z is None else z.double() for z in (x, t, gy, gt))
    w, table = (None if z is None else z.double() for z in (w, table))
    leaves = [x.clone().requires_grad_()]
    if w is not None:
        w = w.clone().requires_grad_()
        leaves.append(w)
    f = lambda z: norm_rope(z, w, table, eps, interleaved)  # noqa: E731
    y = f(leaves[0])
    loss, dy = (y * gy).sum(), None
    if t is not None:
        t = t.clone().requires_grad_()
        leaves.append(t)
        z = torch.zeros_like(y).requires_grad_()
        back, = torch.autograd.grad((y * z).sum(), leaves[0], create_graph=True)
        dy, = torch.autograd.grad((back * t).sum(), z, create_graph=True)
        loss = loss + (dy * gt).sum()
    g = torch.autograd.grad(loss, leaves, allow_unused=True)
    g = [torch.zeros_like(z) if x is None else x for x, z in zip(g, leaves)]
    return {"y": y.detach(), "dy": None if dy is None else dy.detach(), "gx": g[0],
            "gdx": g[-1] if t is not None else None, "gw": g[1] if w is not None else None}


def check_side(got, x, t, gy, gt, w, table, eps, interleaved):
    """Asserts that got (a dict of the same names) is within the bounds."""
    want = side_64(x, t, gy, gt, w, table, eps, interleaved)
    d = lambda z: None if z is None else z.double()  # noqa: E731
    mag = magnitudes(d(x), d(t), d(gy), d(gt), d(w), d(table), eps, interleaved)
    D = x.shape[-1]
    # r, up to three of them in a term; a mean's D products and sums, two means in a
    # term; a dozen products and sums
    steps = (3 * (D / 2 + 8) + 2 * (D + 2) + 12) * S
    for name, value in got.items():
        if value is None:
            continue
        v = value.double().cpu()
        b = steps * mag[name]
        if name == "gw":
            b = b + (mag["rows"] + 2) * S * mag[name]  # sums over rows in any order
        else:
            info = torch.finfo(value.dtype)
            b = b + info.eps / 2 * want[name].abs() + info.smallest_normal * info.eps
        err = (v - want[name]).abs()
        assert (err <= b).all(), (name, (err - b).max().item(), err.max().item())
