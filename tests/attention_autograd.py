"""Derivatives of autograd.jvp_attention, by itself and behind autograd.norm_rope, where only
some of its arguments have tangents (the ways of rope_autograd.py).

`plain_kernels` stands in for the kernels of attention without a GPU.
"""

import concurrent.futures

import rope_autograd as ra
import torch
import torch.autograd.forward_ad as fwAD
from forward_mode_flash_gb300 import api, autograd

B, H, N, D = 2, 2, 5, 16
NAMES = ("q", "k", "v")
SOME = [w for w in ra.SOME if 3 not in w]
MORE_NAMES = ("q", "k", "v", "wq", "wk")
MORE = [(0,), (1,), (2,), (3,), (0, 4), (1, 2), (0, 1, 2, 3, 4)]
_thread = concurrent.futures.ThreadPoolExecutor(1)  # (without the caller's torch.func levels)


def attend(q, k, v, causal):
    """Scores and outputs."""
    s = q @ k.transpose(-1, -2) * D ** -0.5
    if causal:
        s = s.masked_fill(torch.ones(N, N, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
    e = s.exp()  # (softmax itself has no second derivatives by dual tensors in torch)
    return s, e / e.sum(-1, keepdim=True) @ v


def dual(q, k, v, dq, dk, dv, causal):
    s = q @ k.transpose(-1, -2) * D ** -0.5
    ds = (dq @ k.transpose(-1, -2) + q @ dk.transpose(-1, -2)) * D ** -0.5
    if causal:
        s = s.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), float("-inf"))
    p = s.softmax(-1)
    mu = (p * ds).sum(-1, keepdim=True)
    return p @ v, (p * (ds - mu)) @ v + p @ dv, s.logsumexp(-1), mu[..., 0]


def plain_kernels(monkeypatch):
    """Through their signatures in api: plain tensors in and out, float64 between."""
    def wide(ts):
        for t in ts:
            if torch._C._functorch.is_functorch_wrapped_tensor(t):
                raise RuntimeError("a tensor without storage")
        with fwAD._set_fwd_grad_enabled(False):
            return [t.detach().double() for t in ts]

    def run(f, *ts):
        return [x.float() for x in _thread.submit(f, *wide(ts)).result()]

    def back(f, count):
        def g(*ts):
            leaves = [t.clone().requires_grad_() for t in ts[:count]]
            out = f(*leaves)
            return torch.autograd.grad(out, leaves, ts[count:count + len(out)])
        return g

    def attention(q, k, v, attn_mask, is_causal, scale, return_lse):
        s, o = run(lambda *x: attend(*x, is_causal), q, k, v)
        return o, s.logsumexp(-1)

    def bwd(q, k, v, o, lse, g, attn_mask, is_causal, scale):
        return run(back(lambda *x: attend(*x, is_causal)[1:], 3), q, k, v, g)

    def fwd_dual(*ts, attn_mask, is_causal, scale, return_stats):
        return tuple(run(lambda *x: dual(*x, is_causal), *ts))

    def bwd_dual(*ts, attn_mask, is_causal, scale):
        return run(back(lambda *x: dual(*x, is_causal)[:2], 6), *ts[:6], *ts[10:])

    for f in (attention, bwd, fwd_dual, bwd_dual):
        monkeypatch.setattr(api, f.__name__, f)


def own(*args):
    return (autograd.jvp_attention(*args, is_causal=True),)


def plain(*args):
    return attend(*args, True)[1:]


def own_behind(table):
    return lambda q, k, v, wq, wk: own(*autograd.norm_rope(q, k, table, None, wq, wk, ra.EPS), v)


def plain_behind(table):
    f = ra.plain(table)
    return lambda q, k, v, wq, wk: plain(*f(q, k, wq, wk), v)


def compare(way, to, which, behind=None):
    """As rope_autograd.compare."""
    g = torch.Generator().manual_seed(len(which))
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    shapes = [(B, H, N, D)] * 3 + ([(D,)] * 2 if behind is not None else [])
    args, tangents = [r(*s) for s in shapes], [r(*s) for s in shapes]
    c = [r(B, H, N, D) for _ in range(2)]
    own_f = own if behind is None else own_behind(to(behind))
    plain_f = plain if behind is None else plain_behind(behind)
    got = way(own_f, *([to(x) for x in z] for z in (args, tangents, c)), which)
    want = way(plain_f, *([x.double() for x in z] for z in (args, tangents, c)), which)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        # fp32 throughout: some three hundred roundings of 2^-24
        a = a.detach().double().cpu()
        assert (a - b).abs().max() <= 2e-5 * max(1.0, b.abs().max())
