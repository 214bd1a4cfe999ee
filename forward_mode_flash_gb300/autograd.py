"""PyTorch autograd / torch.func integration over the C ABI.

Mirrors the "JVP Flash Attention" project page (Usage section):

* ``JVPAttn.fwd_dual(q, k, v, attn_mask=None, is_causal=False, scale=None)``
  is the call a model makes inside ``torch.func.jvp(model, (x,), (gt,))``.
  When q, k, v carry forward-mode tangents of the innermost jvp level, one
  fused ``fwd_dual`` launch computes O and tO (no separate primal pass), and
  both are returned differentiable: the reverse mode through them runs
  ``bwd_dual``, so a loss of (O, tO) trains through the JVP and the gradient
  of the tangent output is a Hessian-vector product (reverse over forward).
  Called with explicit tangents, ``JVPAttn.fwd_dual(q, k, v, dq, dk, dv)``
  returns (O, tO) from the same fused call.
* ``jvp_attention(q, k, v, attn_mask=None, is_causal=False, scale=None)`` is a
  drop-in for ``scaled_dot_product_attention``.  Under ``torch.func.jvp`` it
  takes the same fused route; elsewhere it is an autograd.Function whose
  forward-mode rule calls ``fwd_dual`` and whose backward calls the
  primal-only ``bwd`` (no tangent terms).

* ``norm_rope(q, k, rope, ...)`` is what comes before attention: norms of
  queries and keys per head and their rotation by position.  Under
  torch.func.jvp one ``norm_rope_dual`` launch gives values and tangents, both
  differentiable; elsewhere it back-propagates through ``norm_rope_bwd``.

All arithmetic runs in the library's kernels; this module only wires them
into autograd.
"""

from __future__ import annotations

from typing import Optional

import torch
import torch.autograd.forward_ad as fwAD

from . import api

_ft = torch._C._functorch


def _zeros_if_none(t, like):
    return torch.zeros_like(like) if t is None else t


def _dense_cotangent(g, like):
    """A storage-backed contiguous cotangent for the kernels.

    Autograd passes None, or a ZeroTensor (a zero without storage, e.g. for
    O when only the tangent output enters the loss), for outputs that do not
    reach the loss."""
    if g is None or g._is_zerotensor():
        return torch.zeros_like(like)
    return g.contiguous()


def _tangents(given, tensors):
    """Tangents that the kernels can read, zeros for none (a zero without storage among
    them); None for tensors that are not there."""
    def usable(t, x):
        if t is None or t._is_zerotensor():
            return torch.zeros_like(x)
        return t if t.stride(-1) == 1 else t.contiguous()
    return tuple(None if x is None else usable(t, x) for t, x in zip(given, tensors))


class _FwdDual(torch.autograd.Function):
    """(O, tO) of one fused fwd_dual call; backward = reverse mode of the dual map."""

    @staticmethod
    def forward(ctx, q, k, v, dq, dk, dv, attn_mask, is_causal, scale):
        o, t_o, lse, mu = api.fwd_dual(q, k, v, dq, dk, dv, attn_mask=attn_mask,
                                       is_causal=is_causal, scale=scale, return_stats=True)
        ctx.save_for_backward(q, k, v, dq, dk, dv, o, t_o, lse, mu)
        ctx.attn_mask, ctx.is_causal, ctx.scale = attn_mask, is_causal, scale
        return o, t_o

    @staticmethod
    def backward(ctx, g_o, g_to):
        q, k, v, dq, dk, dv, o, t_o, lse, mu = ctx.saved_tensors
        g_o = _dense_cotangent(g_o, o)
        g_to = _dense_cotangent(g_to, t_o)
        grads = api.bwd_dual(q, k, v, dq, dk, dv, o, t_o, lse, mu, g_o, g_to,
                             attn_mask=ctx.attn_mask, is_causal=ctx.is_causal, scale=ctx.scale)
        return (*grads, None, None, None)


def _record(function, *args):
    """Applies an autograd.Function at the enclosing level of torch.func.

    functorch's dispatch is off, and the single-level Function is applied
    directly (torch.func would otherwise insist on handling the Function at this
    level itself)."""
    prev = _ft.get_single_level_autograd_function_allowed()
    _ft.set_single_level_autograd_function_allowed(True)
    try:
        with torch._C._DisableFuncTorch():
            return super(torch.autograd.Function, function).apply(*args)
    finally:
        _ft.set_single_level_autograd_function_allowed(prev)


def _fused_under_jvp(q, k, v, attn_mask, is_causal, scale):
    """O as a forward-mode dual (O, tO) from one fused call, or None.

    Applies when any of q, k, v is a torch.func wrapper of the innermost transform
    level that carries a forward-mode tangent there (the body of torch.func.jvp);
    what is of no level is taken as it is, without a tangent.  The primals and
    tangents are unwrapped to the enclosing level's tensors, one _FwdDual node is
    recorded in that level's autograd graph (so O and tO are differentiable through
    bwd_dual), and O and tO are wrapped back as the dual output of this level.
    Anything else (no transform, other transforms such as vmap at this level, jvp
    nested in another transform) returns None.
    """
    level = _ft.maybe_current_level()
    if level is None:
        return None

    def here(x):
        return _ft.is_functorch_wrapped_tensor(x) and _ft.maybe_get_level(x) == level

    def one_level(t):  # the enclosing level's tensor (must be a plain one)
        return _ft.get_unwrapped(t) if here(t) else t

    pairs = [fwAD.unpack_dual(x) if here(x) else (x, None) for x in (q, k, v)]
    if all(t is None for _, t in pairs):
        return None
    ps = [one_level(p) for p, _ in pairs]
    ts = [torch.zeros_like(p) if t is None else one_level(t) for p, (_, t) in zip(ps, pairs)]
    mask = None if attn_mask is None else one_level(attn_mask)
    if any(_ft.is_functorch_wrapped_tensor(t) for t in (*ps, *ts) + ((mask,) if mask is not None else ())):
        return None  # nested transforms: the generic forward-mode rule handles them
    o, t_o = _record(_FwdDual, *ps, *ts, mask, is_causal, scale)
    return fwAD.make_dual(_ft._wrap_for_grad(o, level), _ft._wrap_for_grad(t_o, level))


class _FwdDualRule(torch.autograd.Function):
    """_FwdDual for the forward-mode rule of JVPAttn, at every level of torch.func: also
    lse and its tangent, which have no gradients."""

    @staticmethod
    def forward(q, k, v, dq, dk, dv, attn_mask, is_causal, scale):
        return api.fwd_dual(q, k, v, dq, dk, dv, attn_mask=attn_mask, is_causal=is_causal,
                            scale=scale, return_stats=True)

    @staticmethod
    def setup_context(ctx, inputs, output):
        ctx.mark_non_differentiable(*output[2:])
        ctx.save_for_backward(*inputs[:6], *output)
        ctx.attn_mask, ctx.is_causal, ctx.scale = inputs[6:]

    @staticmethod
    def jvp(ctx, *_):
        raise RuntimeError("jvp_attention: tangents of tangents are not supported")

    @staticmethod
    def backward(ctx, g_o, g_to, *_):
        return _FwdDual.backward(ctx, g_o, g_to)


class JVPAttn(torch.autograd.Function):
    """Attention with a forward-mode rule backed by the fused fwd_dual kernel."""

    @staticmethod
    def forward(q, k, v, attn_mask, is_causal, scale):
        o, lse = api.attention(q, k, v, attn_mask=attn_mask, is_causal=is_causal, scale=scale,
                               return_lse=True)
        return o, lse

    @staticmethod
    def setup_context(ctx, inputs, output):
        q, k, v, attn_mask, is_causal, scale = inputs
        o, lse = output
        ctx.save_for_forward(q, k, v, o, lse)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.attn_mask, ctx.is_causal, ctx.scale = attn_mask, is_causal, scale

    @staticmethod
    def jvp(ctx, dq, dk, dv, *_):
        # (Reached for forward-mode AD that the fused route above does not take, e.g.
        # torch.autograd's forward_ad dual tensors; by a function again, so that the
        # tangent has a history at every level.)
        q, k, v = ctx.saved_tensors[:3]
        _, t_o, _, mu = _FwdDualRule.apply(q, k, v, *_tangents((dq, dk, dv), (q, k, v)),
                                           ctx.attn_mask, ctx.is_causal, ctx.scale)
        return t_o, mu  # mu is the tangent of lse

    @staticmethod
    def backward(ctx, g_o, _g_lse):
        # The primal-only backward (no tangent terms); lse is an auxiliary
        # output whose cotangent is not propagated.
        q, k, v, o, lse = ctx.saved_tensors
        g = api.bwd(q, k, v, o, lse, _dense_cotangent(g_o, o), attn_mask=ctx.attn_mask,
                    is_causal=ctx.is_causal, scale=ctx.scale)
        return g[0], g[1], g[2], None, None, None

    @staticmethod
    def fwd_dual(q, k, v, dq=None, dk=None, dv=None, attn_mask: Optional[torch.Tensor] = None,
                 is_causal: bool = False, scale: Optional[float] = None):
        """Attention whose forward-mode tangent comes from one fused pass.

        ``JVPAttn.fwd_dual(q, k, v)`` (the project page's form): inside
        torch.func.jvp returns O carrying its tangent tO, both from one fused
        launch and both differentiable through bwd_dual; outside any
        transform it is ``jvp_attention(q, k, v)``.

        ``JVPAttn.fwd_dual(q, k, v, dq, dk, dv)``: (O, tO) for explicit
        tangents (None = zero) from one fused launch, differentiable through
        bwd_dual with respect to all six inputs.
        """
        if dq is None and dk is None and dv is None:
            return jvp_attention(q, k, v, attn_mask=attn_mask, is_causal=is_causal, scale=scale)
        dq, dk, dv = (_zeros_if_none(t, x) for t, x in ((dq, q), (dk, k), (dv, v)))
        return _FwdDual.apply(q, k, v, dq, dk, dv, attn_mask, is_causal, scale)


def jvp_attention(q, k, v, attn_mask: Optional[torch.Tensor] = None, is_causal: bool = False,
                  scale: Optional[float] = None) -> torch.Tensor:
    """Drop-in for scaled_dot_product_attention with a fused forward-mode rule."""
    fused = _fused_under_jvp(q, k, v, attn_mask, is_causal, scale)
    if fused is not None:
        return fused
    o, _ = JVPAttn.apply(q, k, v, attn_mask, is_causal, scale)
    return o


# ---- norms of queries and keys, and rotation
def _weight_grads(g, weights):
    return tuple(None if w is None else x.to(w.dtype) for x, w in zip(g, weights))


def _weight_tangents(given, weights):
    """Tangents of both weights, or of none."""
    return (None, None) if all(t is None for t in given) else _tangents(given, weights)


def _run(function, *args):
    """function.apply, without its cost where nothing can differentiate the result."""
    if torch.is_grad_enabled() or _ft.maybe_current_level() is not None or fwAD._current_level >= 0:
        return function.apply(*args)
    return function.forward(*args)


def _wide(*tensors):
    return [x.float() for x in tensors]


class _NormRopeDualGrads(torch.autograd.Function):
    """Gradients of _NormRopeDual's results for cotangents g."""

    @staticmethod
    def forward(q, k, dq, dk, q_weight, k_weight, dq_weight, dk_weight, rope, positions, eps,
                interleaved, *g):
        g = [_dense_cotangent(x, like) for x, like in zip(g, (q, k, q, k))]
        w, dw, options = (q_weight, k_weight), (dq_weight, dk_weight), (eps, interleaved)
        if dq_weight is None:
            out = api.norm_rope_bwd_dual(q, k, dq, dk, *g, rope, positions, *w, *options)
            return (*out[:4], *_weight_grads(out[4:], w), None, None)
        rows, g = _wide(q, k, dq, dk), _wide(*g)
        out = api.norm_rope_bwd_dual(*rows, *g, rope, positions, *w, *options)
        more = api.norm_rope_bwd(*rows[:2], *g[2:], rope, positions, *dw, *options)
        out = (*(x + y for x, y in zip(out[:2], more)), *out[2:])
        return (*(x.to(q.dtype) for x in out[:4]), *_weight_grads(out[4:], w),
                *_weight_grads(more[2:], dw))

    @staticmethod
    def setup_context(ctx, inputs, output):
        pass

    @staticmethod
    def jvp(ctx, *_):
        raise RuntimeError("norm_rope: gradients of tangents have no tangents of their own (with "
                           "torch.autograd.forward_ad, call backward behind the dual_level)")

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("norm_rope is once_differentiable: its gradients have none of their own")


class _NormRopeDual(torch.autograd.Function):
    """(q, k, dq, dk) of one norm_rope_dual call; backward = reverse mode of the dual map.

    Tangents of the weights (None: none): the outputs are linear in the weights, so a
    second call that has these for weights gives what they add.  Both take 16-bit
    rows in 32 bits then, so that the sums are rounded once."""

    @staticmethod
    def forward(q, k, dq, dk, q_weight, k_weight, dq_weight, dk_weight, rope, positions, eps,
                interleaved):
        w, dw, options = (q_weight, k_weight), (dq_weight, dk_weight), (eps, interleaved)
        if dq_weight is None:
            return api.norm_rope_dual(q, k, dq, dk, rope, positions, *w, *options)
        rows = _wide(q, k, dq, dk)
        y = api.norm_rope_dual(*rows, rope, positions, *w, *options)
        more = api.norm_rope(*rows[:2], rope, positions, *dw, *options)
        if q.dtype == torch.float32:
            values = y[:2]
        else:
            values = api.norm_rope(q, k, rope, positions, *w, *options)
        return (*values, *((x + z).to(q.dtype) for x, z in zip(y[2:], more)))

    @staticmethod
    def setup_context(ctx, inputs, output):
        ctx.save_for_forward(*inputs[:10])
        ctx.save_for_backward(*inputs[:10])
        ctx.options = inputs[10:]

    @staticmethod
    def jvp(ctx, *_):
        raise RuntimeError("norm_rope: tangents of tangents are not supported")

    @staticmethod
    def backward(ctx, *g):
        return (*_run(_NormRopeDualGrads, *ctx.saved_tensors, *ctx.options, *g), None, None, None,
                None)


class _NormRopeGrads(torch.autograd.Function):
    """Gradients of _NormRope's results for cotangents g."""

    @staticmethod
    def forward(q, k, q_weight, k_weight, rope, positions, eps, interleaved, *g):
        g = [_dense_cotangent(x, like) for x, like in zip(g, (q, k))]
        out = api.norm_rope_bwd(q, k, *g, rope, positions, q_weight, k_weight, eps, interleaved)
        return (*out[:2], *_weight_grads(out[2:], (q_weight, k_weight)))

    @staticmethod
    def setup_context(ctx, inputs, output):
        ctx.save_for_forward(*inputs[:6], *inputs[8:])
        ctx.options = inputs[6:8]

    @staticmethod
    def jvp(ctx, dq, dk, dqw, dkw, _rope, _positions, _eps, _interleaved, *dg):
        # The gradients are those of <g, y>, so their tangents are the gradients of
        # <dg, y> + <g, dy> by the same tensors.
        q, k, q_weight, k_weight, rope, positions, *g = ctx.saved_tensors
        w = q_weight, k_weight
        out = _NormRopeDualGrads.apply(q, k, *_tangents((dq, dk), (q, k)), *w,
                                       *_weight_tangents((dqw, dkw), w), rope, positions,
                                       *ctx.options, *_tangents((*dg, *g), (q, k, q, k)))
        return (*out[:2], *out[4:6])

    backward = _NormRopeDualGrads.backward


class _NormRope(torch.autograd.Function):
    """norm_rope with a forward-mode rule backed by norm_rope_dual."""

    @staticmethod
    def forward(q, k, q_weight, k_weight, rope, positions, eps, interleaved):
        return api.norm_rope(q, k, rope, positions, q_weight, k_weight, eps, interleaved)

    @staticmethod
    def setup_context(ctx, inputs, output):
        ctx.save_for_forward(*inputs[:6])
        ctx.save_for_backward(*inputs[:6])
        ctx.options = inputs[6:]

    @staticmethod
    def jvp(ctx, dq, dk, dqw, dkw, *_):
        # (by a function again, so that the tangents have a history at every level)
        q, k, q_weight, k_weight, rope, positions = ctx.saved_tensors
        w = q_weight, k_weight
        return _NormRopeDual.apply(q, k, *_tangents((dq, dk), (q, k)), *w,
                                   *_weight_tangents((dqw, dkw), w), rope, positions,
                                   *ctx.options)[2:]

    @staticmethod
    def backward(ctx, *g):
        return (*_run(_NormRopeGrads, *ctx.saved_tensors, *ctx.options, *g), None, None, None, None)


def _norm_rope_under_jvp(q, k, q_weight, k_weight, rope, positions, eps, interleaved):
    """(q, k) as forward-mode duals from one fused call, or None (see _fused_under_jvp).

    Any of q, k and the weights may carry a tangent at this level; what is of no level
    is taken as it is.  What is of another one is left to the generic rule."""
    level = _ft.maybe_current_level()
    if level is None:
        return None

    def here(x):
        return _ft.is_functorch_wrapped_tensor(x) and _ft.maybe_get_level(x) == level

    def one_level(t):
        return _ft.get_unwrapped(t) if t is not None and here(t) else t

    xs = (q, k, q_weight, k_weight)
    pairs = [fwAD.unpack_dual(x) if x is not None and here(x) else (x, None) for x in xs]
    if all(t is None for _, t in pairs):
        return None
    ps, ts = ([one_level(x[i]) for x in pairs] for i in (0, 1))
    rest = (one_level(rope), one_level(positions))
    if any(t is not None and _ft.is_functorch_wrapped_tensor(t) for t in (*ps, *ts, *rest)):
        return None  # nested transforms: the generic forward-mode rule handles them
    with torch._C._DisableFuncTorch():
        d, dw = _tangents(ts[:2], ps[:2]), _weight_tangents(ts[2:], ps[2:])
    y = _record(_NormRopeDual, *ps[:2], *d, *ps[2:], *dw, *rest, eps, interleaved)
    return tuple(fwAD.make_dual(_ft._wrap_for_grad(o, level), _ft._wrap_for_grad(t, level))
                 for o, t in zip(y[:2], y[2:]))


def norm_rope(q, k, rope: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
              q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
              eps: float = 1e-6, interleaved: bool = False):
    """Differentiable ``api.norm_rope``: (q, k), for ``jvp_attention``.

    With forward-mode tangents of any of q, k and the norm weights the outputs carry
    theirs (inside torch.func.jvp from one fused pass), and values and tangents are
    differentiable with respect to q, k, the norm weights and their tangents (rope and
    positions are constants).  Gradients may have tangents, but no gradients of their
    own: what would need these raises, as do tangents of tangents."""
    fused = _norm_rope_under_jvp(q, k, q_weight, k_weight, rope, positions, eps, interleaved)
    if fused is not None:
        return fused
    return _NormRope.apply(q, k, q_weight, k_weight, rope, positions, eps, interleaved)
