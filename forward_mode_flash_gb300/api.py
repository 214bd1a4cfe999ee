"""Python binding of the C ABI: argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
allocates the output tensors with PyTorch, reads pointers, strides and the
current stream, and calls the entry points declared in ``include/jvp_attn.h``.

API shaped after the "JVP Flash Attention" project page (Usage section):
``attention(q, k, v, attn_mask=...)`` is the forward, and ``fwd_dual`` returns
the output together with its tangent for tangents (dq, dk, dv), as
``JVPAttn.fwd_dual`` does under ``torch.func.jvp``.
"""

from __future__ import annotations

import ctypes
import math
import operator
from typing import Optional, Tuple

import torch

from . import _abi

_DT = {torch.float32: _abi.JVP_F32, torch.float16: _abi.JVP_F16, torch.bfloat16: _abi.JVP_BF16}


def _strides(t: torch.Tensor) -> _abi.Strides:
    sb, sh, sn, sd = t.stride()
    return _abi.Strides(sb, sh, sn, sd)


_KV_NAMES = frozenset(("k", "v", "dk", "dv"))


def _check_inputs(tensors, names) -> int:
    """Checks dtype, device, rank and sizes; returns the key/value head count.

    Key-side tensors (k, v, dk, dv) may have fewer heads than the queries
    (grouped-query attention) as long as the query heads are a multiple.
    """
    ref = tensors[0]
    if ref.dim() != 4:
        raise ValueError(f"{names[0]} must be [B, H, N, D], got {tuple(ref.shape)}")
    if ref.dtype not in _DT:
        raise TypeError(f"unsupported dtype {ref.dtype}")
    if ref.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    H = ref.shape[1]
    hkv = next((t.shape[1] for t, n in zip(tensors, names) if n in _KV_NAMES and t.dim() == 4), H)
    if hkv <= 0 and H > 0 or (hkv > 0 and H % hkv != 0):
        raise ValueError(f"query heads ({H}) must be a multiple of key/value heads ({hkv})")
    for t, n in zip(tensors, names):
        if t.dtype != ref.dtype or t.device != ref.device or t.dim() != 4:
            raise ValueError(f"{n} must be a 4-D {ref.dtype} tensor on {ref.device}")
        heads = hkv if n in _KV_NAMES else H
        if t.shape[-1] != ref.shape[-1] or t.shape[0] != ref.shape[0] or t.shape[1] != heads:
            raise ValueError(f"{n} has shape {tuple(t.shape)}, inconsistent with {tuple(ref.shape)}")
        if t.stride(-1) != 1 and t.numel() > 0:
            raise ValueError(f"{n} must have a unit innermost stride")
    return hkv


def _mask_desc(attn_mask: Optional[torch.Tensor], is_causal: bool, B, H, Nq, Nk, device):
    """Mask description (and the tensor it points into, kept alive by the caller).

    ``is_causal`` together with ``attn_mask`` keeps a key only where both do
    (an extension: scaled_dot_product_attention rejects the combination).
    """
    if attn_mask is None:
        kind = _abi.JVP_MASK_CAUSAL if is_causal else _abi.JVP_MASK_NONE
        return _abi.Mask(kind, None, 0, 0, 0, 0), None
    if attn_mask.device != device:
        raise ValueError("attn_mask must be on the same device as q")
    if attn_mask.dtype == torch.bool:
        kind, m = _abi.JVP_MASK_BOOL, attn_mask.view(torch.uint8)
        if is_causal:
            kind = _abi.JVP_MASK_BOOL_CAUSAL
    elif attn_mask.dtype == torch.float32:
        kind, m = _abi.JVP_MASK_ADDITIVE, attn_mask
        if is_causal:
            kind = _abi.JVP_MASK_ADDITIVE_CAUSAL
    else:
        raise TypeError("attn_mask must be torch.bool (keep-mask) or torch.float32 (additive)")
    while m.dim() < 4:
        m = m.unsqueeze(0)
    m = m.expand(B, H, Nq, Nk)  # broadcast dimensions get stride 0
    sb, sh, sq, sk = m.stride()
    return _abi.Mask(kind, m.data_ptr(), sb, sh, sq, sk), m


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def fwd_dual(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dq: torch.Tensor,
             dk: torch.Tensor, dv: torch.Tensor, attn_mask: Optional[torch.Tensor] = None,
             is_causal: bool = False, scale: Optional[float] = None, return_stats: bool = False,
             out: Optional[Tuple[torch.Tensor, ...]] = None, split_kv: bool = True,
             workspace: Optional[torch.Tensor] = None):
    """Attention forward and its JVP in one fused pass.

    Returns (o, t_o), or (o, t_o, lse, mu) with ``return_stats``: lse is the
    natural-log log-sum-exp per row and mu its tangent, both float32 [B,H,Nq].
    ``out`` = (o, t_o) or (o, t_o, lse, mu) gives preallocated outputs (the
    four-tuple implies ``return_stats``).  With ``split_kv`` (the default),
    problems with fewer query tiles than SMs split their key range over
    several CTAs through ``jvp_attn_fwd_dual_ws``; the scratch it needs
    (``fwd_dual_workspace_size``) is allocated here unless ``workspace`` (a
    16-byte-aligned uint8 device tensor) is given.
    """
    lib = _abi.load()
    if attn_mask is None and out is None and workspace is None:
        plan = _fwd_plan(lib, q, k, v, dq, dk, dv, is_causal, split_kv)
        if plan is not None:
            return _fwd_dual_planned(lib, plan, q, k, v, dq, dk, dv, scale, return_stats)
    hkv = _check_inputs([q, k, v, dq, dk, dv], ["q", "k", "v", "dq", "dk", "dv"])
    B, H, Nq, D = q.shape
    Nk = k.shape[2]
    for t, n in ((v, "v"), (dk, "dk"), (dv, "dv")):
        if t.shape[2] != Nk:
            raise ValueError(f"{n} must have {Nk} rows")
    if dq.shape[2] != Nq:
        raise ValueError("dq must match q")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        o = torch.empty((B, H, Nq, D), dtype=q.dtype, device=q.device)
        t_o = torch.empty_like(o)
    else:
        o, t_o = out[0], out[1]
    if out is not None and len(out) == 4:
        lse, mu = out[2], out[3]
        for t, n in ((lse, "lse"), (mu, "mu")):
            if (t.dtype != torch.float32 or tuple(t.shape) != (B, H, Nq) or not t.is_contiguous()
                    or t.device != q.device):
                raise ValueError(f"out {n} must be a contiguous float32 [B, H, Nq] device tensor")
        return_stats = True
    else:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if return_stats else None
        mu = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if return_stats else None
    mask, _keep = _mask_desc(attn_mask, is_causal, B, H, Nq, Nk, q.device)
    ins = (_abi.Strides * 6)(*[_strides(t) for t in (q, k, v, dq, dk, dv)])
    outs = (_abi.Strides * 2)(_strides(o), _strides(t_o))
    shape = _abi.Shape(B, H, Nq, Nk, D, hkv)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        need = _split_ws_bytes(lib, shape, q) if split_kv else 0
        if need > 0:
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            st = lib.jvp_attn_fwd_dual_ws(ctypes.byref(shape), _DT[q.dtype], _ptr(q), _ptr(k),
                                          _ptr(v), _ptr(dq), _ptr(dk), _ptr(dv), ins,
                                          ctypes.byref(mask), float(scale), _ptr(o), _ptr(t_o),
                                          outs, _ptr(lse), _ptr(mu), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          ctypes.c_void_p(stream))
        else:
            st = lib.jvp_attn_fwd_dual(ctypes.byref(shape), _DT[q.dtype], _ptr(q), _ptr(k),
                                       _ptr(v), _ptr(dq), _ptr(dk), _ptr(dv), ins,
                                       ctypes.byref(mask), float(scale), _ptr(o), _ptr(t_o),
                                       outs, _ptr(lse), _ptr(mu), ctypes.c_void_p(stream))
    _abi.check(st)
    if return_stats:
        return o, t_o, lse, mu
    return o, t_o


# Validated call descriptions for repeated fwd_dual calls on tensors of the
# same dtypes, devices, shapes and strides (no mask tensor, fresh outputs):
# the ctypes records are built once and only the pointers change per call.
_FWD_PLANS = {}
_FWD_PLANS_MAX = 256


class _FwdPlan:
    __slots__ = ("shape", "ins", "outs", "mask", "dt", "need", "oshape", "sshape", "scale",
                 "dtype", "device", "dev_index")


def _fwd_plan(lib, q, k, v, dq, dk, dv, is_causal, split_kv):
    ts = (q, k, v, dq, dk, dv)
    key = (tuple((t.dtype, t.device, t.shape, t.stride()) for t in ts), bool(is_causal),
           bool(split_kv))
    plan = _FWD_PLANS.get(key)
    if plan is not None:
        return plan
    hkv = _check_inputs(list(ts), ["q", "k", "v", "dq", "dk", "dv"])
    B, H, Nq, D = q.shape
    Nk = k.shape[2]
    if v.shape[2] != Nk or dk.shape[2] != Nk or dv.shape[2] != Nk or dq.shape[2] != Nq:
        return None  # the general path reports the mismatch
    plan = _FwdPlan()
    plan.shape = _abi.Shape(B, H, Nq, Nk, D, hkv)
    plan.ins = (_abi.Strides * 6)(*[_strides(t) for t in ts])
    # outputs are allocated contiguous [B, H, Nq, D]
    plan.outs = (_abi.Strides * 2)(*[_abi.Strides(H * Nq * D, Nq * D, D, 1)] * 2)
    plan.mask = _abi.Mask(_abi.JVP_MASK_CAUSAL if is_causal else _abi.JVP_MASK_NONE, None,
                          0, 0, 0, 0)
    plan.dt = _DT[q.dtype]
    plan.dtype, plan.device, plan.dev_index = q.dtype, q.device, q.device.index
    plan.oshape, plan.sshape = (B, H, Nq, D), (B, H, Nq)
    plan.scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        plan.need = _split_ws_bytes(lib, plan.shape, q) if split_kv else 0
    if len(_FWD_PLANS) >= _FWD_PLANS_MAX:
        _FWD_PLANS.clear()
    _FWD_PLANS[key] = plan
    return plan


def _fwd_dual_planned(lib, plan, q, k, v, dq, dk, dv, scale, return_stats):
    dev = plan.device
    o = torch.empty(plan.oshape, dtype=plan.dtype, device=dev)
    t_o = torch.empty(plan.oshape, dtype=plan.dtype, device=dev)
    lse = mu = None
    if return_stats:
        lse = torch.empty(plan.sshape, dtype=torch.float32, device=dev)
        mu = torch.empty(plan.sshape, dtype=torch.float32, device=dev)
    sc = plan.scale if scale is None else float(scale)
    guard = torch.cuda.current_device() != plan.dev_index
    if guard:
        ctx = torch.cuda.device(dev)
        ctx.__enter__()
    try:
        stream = torch.cuda.current_stream(plan.dev_index).cuda_stream
        lp = lse.data_ptr() if lse is not None else None
        mp = mu.data_ptr() if mu is not None else None
        if plan.need > 0:
            ws = torch.empty(plan.need, dtype=torch.uint8, device=dev)
            st = lib.jvp_attn_fwd_dual_ws(ctypes.byref(plan.shape), plan.dt, q.data_ptr(),
                                          k.data_ptr(), v.data_ptr(), dq.data_ptr(),
                                          dk.data_ptr(), dv.data_ptr(), plan.ins,
                                          ctypes.byref(plan.mask), sc, o.data_ptr(),
                                          t_o.data_ptr(), plan.outs, lp, mp, ws.data_ptr(),
                                          plan.need, stream)
        else:
            st = lib.jvp_attn_fwd_dual(ctypes.byref(plan.shape), plan.dt, q.data_ptr(),
                                       k.data_ptr(), v.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                       dv.data_ptr(), plan.ins, ctypes.byref(plan.mask), sc,
                                       o.data_ptr(), t_o.data_ptr(), plan.outs, lp, mp, stream)
    finally:
        if guard:
            ctx.__exit__(None, None, None)
    _abi.check(st)
    if return_stats:
        return o, t_o, lse, mu
    return o, t_o


_split_ws_cache = {}


def _split_ws_bytes(lib, shape, q) -> int:
    """jvp_attn_fwd_dual_workspace_size, cached per device and shape."""
    key = (q.device.index, shape.B, shape.H, shape.Nq, shape.Nk, shape.D, q.dtype)
    need = _split_ws_cache.get(key)
    if need is None:
        need = int(lib.jvp_attn_fwd_dual_workspace_size(ctypes.byref(shape), _DT[q.dtype]))
        _split_ws_cache[key] = need
    return need


def fwd_dual_workspace_size(B: int, H: int, Nq: int, Nk: int, D: int,
                            dtype: torch.dtype = torch.bfloat16, Hkv: int = 0) -> int:
    """Bytes of scratch with which fwd_dual splits the key range (0: no split)."""
    shape = _abi.Shape(B, H, Nq, Nk, D, Hkv)
    return int(_abi.load().jvp_attn_fwd_dual_workspace_size(ctypes.byref(shape), _DT[dtype]))


def fwd_dual_host_workspace_size(B: int, H: int, Nq: int, Nk: int, D: int,
                                 dtype: torch.dtype = torch.bfloat16, chunks: int = 4) -> int:
    """Device staging bytes of fwd_dual_host for this shape and chunk count."""
    shape = _abi.Shape(B, H, Nq, Nk, D, 0)
    return int(_abi.load().jvp_attn_fwd_dual_host_workspace_size(ctypes.byref(shape),
                                                                 _DT[dtype], int(chunks)))


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              attn_mask: Optional[torch.Tensor] = None, is_causal: bool = False,
              scale: Optional[float] = None, return_lse: bool = False,
              out: Optional[torch.Tensor] = None):
    """Attention forward only (no tangents): o, or (o, lse) with ``return_lse``."""
    lib = _abi.load()
    hkv = _check_inputs([q, k, v], ["q", "k", "v"])
    B, H, Nq, D = q.shape
    Nk = k.shape[2]
    if v.shape[2] != Nk:
        raise ValueError("v must match k")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    o = torch.empty((B, H, Nq, D), dtype=q.dtype, device=q.device) if out is None else out
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if return_lse else None
    mask, _keep = _mask_desc(attn_mask, is_causal, B, H, Nq, Nk, q.device)
    ins = (_abi.Strides * 3)(*[_strides(t) for t in (q, k, v)])
    outs = (_abi.Strides * 1)(_strides(o))
    shape = _abi.Shape(B, H, Nq, Nk, D, hkv)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        st = lib.jvp_attn_fwd(ctypes.byref(shape), _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), ins,
                              ctypes.byref(mask), float(scale), _ptr(o), outs, _ptr(lse),
                              ctypes.c_void_p(stream))
    _abi.check(st)
    return (o, lse) if return_lse else o


def bwd_dual_workspace_size(B: int, H: int, Nq: int, Nk: int, D: int,
                            dtype: torch.dtype = torch.bfloat16, hkv: int = 0) -> int:
    """Bytes of device scratch jvp_attn_bwd_dual needs for this shape on the
    current device (``hkv``: key/value heads, 0 = H)."""
    shape = _abi.Shape(B, H, Nq, Nk, D, hkv)
    return int(_abi.load().jvp_attn_bwd_dual_workspace_size(ctypes.byref(shape), _DT[dtype]))


def bwd_dual(q, k, v, dq, dk, dv, o, t_o, lse, mu, g_o, g_to,
             attn_mask: Optional[torch.Tensor] = None, is_causal: bool = False,
             scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of <g_o, O> + <g_to, tO> with respect to (q, k, v, dq, dk, dv).

    o, t_o, lse, mu are the outputs of ``fwd_dual(..., return_stats=True)`` on
    the same inputs.  ``workspace`` (uint8, on q's device) is allocated here if
    not given; its size is ``bwd_dual_workspace_size``.
    """
    lib = _abi.load()
    hkv = _check_inputs([q, k, v, dq, dk, dv, o, t_o, g_o, g_to],
                        ["q", "k", "v", "dq", "dk", "dv", "o", "t_o", "g_o", "g_to"])
    B, H, Nq, D = q.shape
    Nk = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    for t, n in ((lse, "lse"), (mu, "mu")):
        if t.dtype != torch.float32 or tuple(t.shape) != (B, H, Nq) or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous float32 [B, H, Nq] tensor")
    outs = [torch.empty_like(x) for x in (q, k, v, dq, dk, dv)]
    need = bwd_dual_workspace_size(B, H, Nq, Nk, D, q.dtype, hkv)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    mask, _keep = _mask_desc(attn_mask, is_causal, B, H, Nq, Nk, q.device)
    ins = (_abi.Strides * 10)(*[_strides(t) for t in (q, k, v, dq, dk, dv, o, t_o, g_o, g_to)])
    ost = (_abi.Strides * 6)(*[_strides(t) for t in outs])
    shape = _abi.Shape(B, H, Nq, Nk, D, hkv)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        st = lib.jvp_attn_bwd_dual(ctypes.byref(shape), _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v),
                                   _ptr(dq), _ptr(dk), _ptr(dv), _ptr(o), _ptr(t_o), _ptr(lse),
                                   _ptr(mu), _ptr(g_o), _ptr(g_to), ins, ctypes.byref(mask),
                                   float(scale), *[_ptr(x) for x in outs], ost, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   ctypes.c_void_p(stream))
    _abi.check(st)
    return tuple(outs)


def bwd_workspace_size(B: int, H: int, Nq: int, Nk: int, D: int,
                       dtype: torch.dtype = torch.bfloat16, hkv: int = 0) -> int:
    """Bytes of device scratch jvp_attn_bwd needs for this shape on the
    current device (``hkv``: key/value heads, 0 = H)."""
    shape = _abi.Shape(B, H, Nq, Nk, D, hkv)
    return int(_abi.load().jvp_attn_bwd_workspace_size(ctypes.byref(shape), _DT[dtype]))


def bwd(q, k, v, o, lse, g_o, attn_mask: Optional[torch.Tensor] = None, is_causal: bool = False,
        scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of <g_o, O> with respect to (q, k, v): the backward of
    attention without tangents.

    o, lse are the outputs of ``attention(..., return_lse=True)`` (or of
    ``fwd_dual``) on the same inputs.  ``workspace`` (uint8, on q's device) is
    allocated here if not given; its size is ``bwd_workspace_size``.
    """
    lib = _abi.load()
    hkv = _check_inputs([q, k, v, o, g_o], ["q", "k", "v", "o", "g_o"])
    B, H, Nq, D = q.shape
    Nk = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, Nq] tensor")
    outs = [torch.empty_like(x) for x in (q, k, v)]
    need = bwd_workspace_size(B, H, Nq, Nk, D, q.dtype, hkv)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    mask, _keep = _mask_desc(attn_mask, is_causal, B, H, Nq, Nk, q.device)
    ins = (_abi.Strides * 5)(*[_strides(t) for t in (q, k, v, o, g_o)])
    ost = (_abi.Strides * 3)(*[_strides(t) for t in outs])
    shape = _abi.Shape(B, H, Nq, Nk, D, hkv)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        st = lib.jvp_attn_bwd(ctypes.byref(shape), _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v),
                              _ptr(o), _ptr(lse), _ptr(g_o), ins, ctypes.byref(mask),
                              float(scale), *[_ptr(x) for x in outs], ost, _ptr(workspace),
                              workspace.numel() * workspace.element_size(),
                              ctypes.c_void_p(stream))
    _abi.check(st)
    return tuple(outs)


def fwd_dual_host(q, k, v, dq, dk, dv, attn_mask: Optional[torch.Tensor] = None,
                  is_causal: bool = False, scale: Optional[float] = None, chunks: int = 4,
                  device=None, out: Optional[Tuple[torch.Tensor, ...]] = None,
                  return_stats: bool = False, workspace: Optional[torch.Tensor] = None):
    """fwd_dual for host-resident tensors through ``jvp_attn_fwd_dual_host``.

    q, k, v, dq, dk, dv are contiguous CPU tensors [B, H, N, D] (pinned memory
    lets the copies overlap the kernels).  The library pipelines the copies in,
    the fused kernel and the copies out over ``chunks`` groups of (batch,
    head) pairs.  Returns CPU tensors (O, tO) (plus lse, mu with
    ``return_stats``), or fills ``out``.  A mask must be shared by every
    (batch, head): [Nq, Nk] or [1, 1, Nq, Nk]; it is copied to the device.
    """
    lib = _abi.load()
    dev = torch.device(device) if device is not None else torch.device("cuda",
                                                                        torch.cuda.current_device())
    B, H, Nq, D = q.shape
    Nk = k.shape[2]
    for t in (q, k, v, dq, dk, dv):
        if t.device.type != "cpu" or not t.is_contiguous() or t.dtype != q.dtype:
            raise ValueError("fwd_dual_host takes contiguous CPU tensors of one dtype")
    if k.shape[1] != H:
        raise ValueError("fwd_dual_host needs as many key/value heads as query heads")
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    mask_d = None
    if attn_mask is not None:
        m = attn_mask
        while m.dim() > 2 and m.shape[0] == 1:
            m = m[0]
        if m.dim() != 2:
            raise ValueError("fwd_dual_host needs a mask shared by all batches and heads")
        mask_d = m.to(dev, non_blocking=True)
    mask, _keep = _mask_desc(mask_d, is_causal, 1, 1, Nq, Nk, dev)
    mask.stride_b = mask.stride_h = 0
    pin = q.is_pinned()
    if out is None:
        o_h = torch.empty((B, H, Nq, D), dtype=q.dtype, pin_memory=pin)
        t_h = torch.empty((B, H, Nq, D), dtype=q.dtype, pin_memory=pin)
        lse_h = torch.empty((B, H, Nq), dtype=torch.float32, pin_memory=pin) if return_stats else None
        mu_h = torch.empty((B, H, Nq), dtype=torch.float32, pin_memory=pin) if return_stats else None
    else:
        o_h, t_h = out[0], out[1]
        lse_h, mu_h = (out[2], out[3]) if len(out) == 4 else (None, None)
    shape = _abi.Shape(B, H, Nq, Nk, D, 0)
    need = int(lib.jvp_attn_fwd_dual_host_workspace_size(ctypes.byref(shape), _DT[q.dtype],
                                                         int(chunks)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    with torch.cuda.device(dev):
        st = lib.jvp_attn_fwd_dual_host(ctypes.byref(shape), _DT[q.dtype], _ptr(q), _ptr(k),
                                        _ptr(v), _ptr(dq), _ptr(dk), _ptr(dv), ctypes.byref(mask),
                                        float(scale), _ptr(o_h), _ptr(t_h), _ptr(lse_h),
                                        _ptr(mu_h), int(chunks), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        ctypes.c_void_p(stream))
    _abi.check(st)
    # keep the staging area and the device mask alive until the stream is done
    workspace.record_stream(torch.cuda.current_stream(dev))
    if mask_d is not None:
        mask_d.record_stream(torch.cuda.current_stream(dev))
    if return_stats or (out is not None and len(out) == 4):
        return o_h, t_h, lse_h, mu_h
    return o_h, t_h


# ---- packed prompts, the paged key-value cache and the attention over it
_E4M3 = torch.float8_e4m3fn
_bind = None  # the binding's native part


def _native(name):
    """The native part of the binding, and the address of an entry point."""
    global _bind
    lib = _abi.load()
    if _bind is None:
        _bind = _abi.load_bind()
    return _bind, lib.addresses[name]


def _check_int32(t, name, shape, device):
    if t.dtype != torch.int32 or t.device != device:
        raise ValueError(f"{name} must be an int32 tensor on {device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have a unit innermost stride")


def _check_packed(t, name, ref_dtype, device, shape):
    if t.dim() != 3 or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be [rows, heads, D] = {shape}, got {tuple(t.shape)}")
    if t.dtype != ref_dtype or t.device != device:
        raise ValueError(f"{name} must be a {ref_dtype} tensor on {device}")
    if t.stride(-1) != 1 and t.numel() > 0:
        raise ValueError(f"{name} must have a unit innermost stride")


def _cache_desc(k_cache, v_cache, block_table, k_scale, v_scale):
    """Checks the tensors of a paged cache; its description for the library."""
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache must be [pages, Hkv, page_size, D], got {tuple(k_cache.shape)}")
    if k_cache.dtype not in _DT and k_cache.dtype != _E4M3:
        raise TypeError(f"unsupported cache dtype {k_cache.dtype}")
    if k_cache.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    dev = k_cache.device
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype or v_cache.device != dev:
        raise ValueError("v_cache must have k_cache's shape, dtype and device")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.stride(-1) != 1 and t.numel() > 0:
            raise ValueError(f"{n} must have a unit innermost stride")
    pages, hkv, page, D = k_cache.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    _check_int32(block_table, "block_table", tuple(block_table.shape), dev)
    if k_cache.dtype == _E4M3:
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if (t is None or t.dtype != torch.uint8 or t.device != dev
                    or tuple(t.shape) != (pages, hkv, page) or not t.is_contiguous()):
                raise ValueError(f"{n} must be a contiguous uint8 [pages, Hkv, page_size] tensor "
                                 "on the cache's device")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to an e4m3 cache only")
    sk, sv = k_cache.stride(), v_cache.stride()
    return _abi.Cache(pages, page, hkv, D, block_table.shape[0], block_table.shape[1],
                      block_table.stride(0),
                      _abi.JVP_E4M3 if k_cache.dtype == _E4M3 else _DT[k_cache.dtype],
                      _abi.Strides(sk[0], sk[1], sk[2], 1), _abi.Strides(sv[0], sv[1], sv[2], 1))


def _check_packed_call(q, k, v, cu_seqlens, out):
    if q.dim() != 3:
        raise ValueError(f"q must be [T, H, D], got {tuple(q.shape)}")
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if q.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    T, H, D = q.shape
    hkv = k.shape[1] if k.dim() == 3 else -1
    if hkv <= 0 and H > 0 or hkv > 0 and H % hkv != 0:
        raise ValueError(f"query heads ({H}) must be a multiple of key/value heads ({hkv})")
    _check_packed(q, "q", q.dtype, q.device, (T, H, D))
    _check_packed(k, "k", q.dtype, q.device, (T, hkv, D))
    _check_packed(v, "v", q.dtype, q.device, (T, hkv, D))
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [B + 1]")
    B = cu_seqlens.shape[0] - 1
    _check_int32(cu_seqlens, "cu_seqlens", (B + 1,), q.device)
    if out is not None:
        _check_packed(out, "out", q.dtype, q.device, (T, H, D))


def attention_packed(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     is_causal: bool = False, scale: Optional[float] = None,
                     return_lse: bool = False, out: Optional[torch.Tensor] = None):
    """Attention over whole prompts of different lengths, packed one behind the other.

    q is [T, H, D], k and v [T, Hkv, D] with H a multiple of Hkv (grouped-query
    attention); sequence b's rows are ``cu_seqlens[b]:cu_seqlens[b + 1]``
    (int32 [B + 1], non-decreasing, on the device, read when the work runs) and
    attend to each other only (``is_causal``: row i to rows j <= i).  Returns o
    [T, H, D], or (o, lse) with ``return_lse`` (float32 [H, T]).  Rows that
    belong to no sequence are not written (give ``out`` to keep what it holds).
    Forward only, as ``attention``: no gradient or tangent passes through.
    """
    bind, entry = _native("jvp_attn_fwd_packed")
    r = bind.packed(entry, q, k, v, cu_seqlens, out, is_causal, scale, return_lse)
    if r is None:  # a layout not seen before
        _check_packed_call(q, k, v, cu_seqlens, out)
        bind.remember(bind.PACKED, 0, q, k, v, cu_seqlens, out)
        r = bind.packed(entry, q, k, v, cu_seqlens, out, is_causal, scale, return_lse)
    if type(r) is int:
        _abi.check(r)
    return r


def _check_rows(k, v, k_cache, v_cache, block_table, start_pos, cu_seqlens, k_scale, v_scale):
    """Checks of cache_write and cache_read, with packed rows k, v."""
    desc = _cache_desc(k_cache, v_cache, block_table, k_scale, v_scale)
    dev = k_cache.device
    if k.dtype not in _DT:
        raise TypeError(f"unsupported dtype {k.dtype}")
    if k_cache.dtype != _E4M3 and k.dtype != k_cache.dtype:
        raise ValueError("k and v must have the cache's dtype (unless the cache is e4m3)")
    shape = (k.shape[0] if k.dim() == 3 else -1, desc.Hkv, desc.D)
    _check_packed(k, "k", k.dtype, dev, shape)
    _check_packed(v, "v", k.dtype, dev, shape)
    if start_pos is not None:
        _check_int32(start_pos, "start_pos", (desc.B,), dev)
    if cu_seqlens is not None:
        _check_int32(cu_seqlens, "cu_seqlens", (desc.B + 1,), dev)
    elif shape[0] != desc.B:
        raise ValueError("without cu_seqlens there must be one row per sequence")


def _rows(write, name, *tensors):
    """cache_write or cache_read: (k, v, k_cache, v_cache, block_table, start_pos,
    cu_seqlens, k_scale, v_scale)."""
    bind, entry = _native(name)
    f = bind.write if write else bind.read
    st = f(entry, *tensors)
    if st is None:  # a layout not seen before
        _check_rows(*tensors)
        bind.remember(bind.WRITE if write else bind.READ, 0, *tensors)
        st = f(entry, *tensors)
    _abi.check(st)


def cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                block_table: torch.Tensor, start_pos: Optional[torch.Tensor] = None,
                cu_seqlens: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                v_scale: Optional[torch.Tensor] = None) -> None:
    """Writes new rows of keys and values into the pages of their sequences.

    k, v are [T, Hkv, D], the new rows of all sequences behind one another:
    sequence b's are ``cu_seqlens[b]:cu_seqlens[b + 1]`` (int32, on the device;
    None: one row per sequence), and go to its positions ``start_pos[b]`` and
    on (int32; None: 0).  Position r is row ``r % page_size`` of page
    ``block_table[b, r // page_size]`` of k_cache, v_cache [pages, Hkv,
    page_size, D].  The cache has k's dtype, or is ``torch.float8_e4m3fn`` with
    one scale byte per (page, head, row) in k_scale, v_scale (uint8 [pages,
    Hkv, page_size]): an entry is ``code * 2**(byte - 127)``, the scale the
    smallest power of two that fits the row's largest magnitude.  Rows that
    belong to no sequence are ignored; rows whose place is out of range, and
    sequences whose offsets decrease or leave [0, T], are skipped
    and reported by ``device_status`` (JVP_ERR_INDEX).  No two rows of a call
    may have the same place.
    """
    _rows(True, "jvp_attn_cache_write", k, v, k_cache, v_cache, block_table, start_pos,
          cu_seqlens, k_scale, v_scale)


def cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
               start_pos: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
               num_rows: Optional[int] = None, k_scale: Optional[torch.Tensor] = None,
               v_scale: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """Rows of the cache back as packed k, v [num_rows, Hkv, D].

    The reverse of ``cache_write``: sequence b's positions ``start_pos[b]`` (None:
    0) and on become rows ``cu_seqlens[b]:cu_seqlens[b + 1]``.  ``num_rows`` is
    the number of rows to allocate, at least ``cu_seqlens[-1]`` (which lives on
    the device); ``out`` = (k, v) gives preallocated ones instead.  Without
    cu_seqlens one row per sequence.  An e4m3 cache's entries become their
    values in ``dtype`` (default bfloat16).  Rows that belong to no sequence,
    and those that ``cache_write`` would skip and report, are not written.
    """
    if out is None:
        if num_rows is None:
            if cu_seqlens is not None:
                raise ValueError("num_rows (or out) is needed with cu_seqlens")
            num_rows = block_table.shape[0]
        k, v = _native("jvp_attn_cache_read")[0].empty_rows(k_cache, num_rows, dtype)
    else:
        k, v = out
        if dtype is not None and k.dtype != dtype:
            raise ValueError(f"out has dtype {k.dtype}, not {dtype}")
    _rows(False, "jvp_attn_cache_read", k, v, k_cache, v_cache, block_table, start_pos,
          cu_seqlens, k_scale, v_scale)
    return k, v


_NO_WINDOW = (1 << 31) - 1  # as wide as any sequence


def _window(window, sinks):
    """Checked window and sinks, as whole numbers."""
    window, sinks = _NO_WINDOW if window is None else operator.index(window), operator.index(sinks)
    if window <= 0 or sinks < 0:
        raise ValueError(f"window must be positive and sinks not negative, got {window} and {sinks}")
    return min(window, _NO_WINDOW), min(sinks, _NO_WINDOW)


def _check_decode(q, k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, out):
    """Checks of attention_decode; the workspace bytes of such a call."""
    desc = _cache_desc(k_cache, v_cache, block_table, k_scale, v_scale)
    dev = k_cache.device
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if k_cache.dtype != _E4M3 and q.dtype != k_cache.dtype:
        raise ValueError("q must have the cache's dtype (unless the cache is e4m3)")
    H = q.shape[1] if q.dim() == 3 else -1
    shape = (desc.B, H, desc.D)
    _check_packed(q, "q", q.dtype, dev, shape)
    if desc.Hkv <= 0 and H > 0 or desc.Hkv > 0 and H % desc.Hkv != 0:
        raise ValueError(f"query heads ({H}) must be a multiple of key/value heads ({desc.Hkv})")
    _check_int32(seq_lens, "seq_lens", (desc.B,), dev)
    if out is not None:
        _check_packed(out, "out", q.dtype, dev, shape)
    with torch.cuda.device(dev):
        return int(_abi.load().jvp_attn_decode_workspace_size(desc, H, _DT[q.dtype]))


def attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_table: torch.Tensor, seq_lens: torch.Tensor,
                     k_scale: Optional[torch.Tensor] = None,
                     v_scale: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     return_lse: bool = False, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, window: Optional[int] = None,
                     sinks: int = 0):
    """Attention of one new token per sequence over its cached keys and values.

    q is [B, H, D]; the cache and block_table are as for ``cache_write`` (which
    puts the token's own row in first, if it is to attend to itself); seq_lens
    (int32 [B], on the device) is the number of positions each sequence
    attends to.  H is a multiple of the cache's heads (grouped-query
    attention).  Returns o [B, H, D], or (o, lse) with ``return_lse`` (float32
    [B, H]); a sequence without keys gets o = 0 and lse = -inf.  ``workspace``
    (uint8, 16-byte aligned, ``decode_workspace_size`` bytes) is allocated here
    if not given; calls that share one must not overlap.  With ``window`` only the
    last ``window`` positions and the first ``sinks`` are attended to, and only these
    are read (block-table entries of others may hold anything).  Forward only, as
    ``attention_packed``.
    """
    if workspace is not None and (workspace.device != k_cache.device
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {k_cache.device}")
    layout = (q, k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, out)
    if window is None and sinks == 0:
        bind, entry = _native("jvp_attn_decode")
        call, rest = bind.decode, (workspace, scale, return_lse)
    else:
        bind, entry = _native("jvp_attn_decode_window")
        call, rest = bind.decode_window, (workspace, *_window(window, sinks), scale, return_lse)
    r = call(entry, *layout, *rest)
    if r is None:  # a layout not seen before
        bind.remember(bind.DECODE, _check_decode(*layout), *layout)
        r = call(entry, *layout, *rest)
    if type(r) is int:
        _abi.check(r)
    return r


def _cache_like(k_cache, block_table):
    """Description of a cache whose values lie as its keys, unchecked."""
    sk = k_cache.stride()
    strides = _abi.Strides(sk[0], sk[1], sk[2], 1)
    pages, hkv, page, D = k_cache.shape
    return _abi.Cache(pages, page, hkv, D, block_table.shape[0], block_table.shape[1],
                      block_table.stride(0),
                      _abi.JVP_E4M3 if k_cache.dtype == _E4M3 else _DT[k_cache.dtype], strides,
                      strides)


def decode_workspace_size(k_cache: torch.Tensor, block_table: torch.Tensor, H: int,
                          dtype: Optional[torch.dtype] = None) -> int:
    """Bytes of scratch that attention_decode needs for H query heads over this
    cache (``dtype``: of the queries; default the cache's, bfloat16 over e4m3)."""
    if dtype is None:
        dtype = torch.bfloat16 if k_cache.dtype == _E4M3 else k_cache.dtype
    desc = _cache_like(k_cache, block_table)
    with torch.cuda.device(k_cache.device):
        return int(_abi.load().jvp_attn_decode_workspace_size(desc, int(H), _DT[dtype]))


def _check_chunk(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, k_scale, v_scale, out):
    """Checks of attention_chunk; the workspace bytes of such a call."""
    desc = _cache_desc(k_cache, v_cache, block_table, k_scale, v_scale)
    dev = k_cache.device
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if k_cache.dtype != _E4M3 and q.dtype != k_cache.dtype:
        raise ValueError("q must have the cache's dtype (unless the cache is e4m3)")
    if q.dim() != 3:
        raise ValueError(f"q must be [T, H, D], got {tuple(q.shape)}")
    T, H = q.shape[:2]
    _check_packed(q, "q", q.dtype, dev, (T, H, desc.D))
    if desc.Hkv <= 0 and H > 0 or desc.Hkv > 0 and H % desc.Hkv != 0:
        raise ValueError(f"query heads ({H}) must be a multiple of key/value heads ({desc.Hkv})")
    _check_int32(seq_lens, "seq_lens", (desc.B,), dev)
    _check_int32(cu_seqlens, "cu_seqlens", (desc.B + 1,), dev)
    if out is not None:
        _check_packed(out, "out", q.dtype, dev, (T, H, desc.D))
    with torch.cuda.device(dev):
        return int(_abi.load().jvp_attn_chunk_workspace_size(desc, H, _DT[q.dtype], T))


def attention_chunk(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_table: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens: torch.Tensor,
                    window: Optional[int] = None, sinks: int = 0,
                    k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    return_lse: bool = False, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None):
    """Attention of some new tokens of each sequence over its cached keys and values.

    q is [T, H, D]; sequence b's new tokens are its rows ``cu_seqlens[b]:cu_seqlens[b +
    1]`` (int32 [B + 1], on the device) and the last of its ``seq_lens[b]`` positions
    (int32 [B], on the device, the new ones included); their keys and values are in the
    cache already (``cache_append`` or ``cache_write``, which also describe the cache
    and block_table).  The token at position x attends to positions j <= x; with
    ``window``, of these to j > x - window and to j < sinks (positions that no new token
    of a sequence attends to are not read, and their block-table entries may hold
    anything).  H is a multiple of the cache's heads (grouped-query attention).
    Returns o [T, H, D], or (o, lse) with ``return_lse`` (float32 [H, T]); a token that
    sees nothing gets o = 0 and lse = -inf, and rows that belong to no sequence are not
    written.  Over an e4m3 cache float16 and bfloat16 queries take its entries as
    ``cache_read`` gives them in that type (float16: infinite beyond 65504, where
    ``attention_decode`` keeps the scale apart).  ``workspace`` as in ``attention_decode``
    (``chunk_workspace_size`` bytes).  Forward only, as ``attention_packed``.
    """
    if workspace is not None and (workspace.device != k_cache.device
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {k_cache.device}")
    bind, entry = _native("jvp_attn_chunk")
    layout = (q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, k_scale, v_scale, out)
    rest = (workspace, *_window(window, sinks), scale, return_lse)
    r = bind.chunk(entry, *layout, *rest)
    if r is None:  # a layout not seen before
        bind.remember(bind.CHUNK, _check_chunk(*layout), *layout)
        r = bind.chunk(entry, *layout, *rest)
    if type(r) is int:
        _abi.check(r)
    return r


def chunk_workspace_size(q: torch.Tensor, k_cache: torch.Tensor, block_table: torch.Tensor) -> int:
    """Bytes of scratch that attention_chunk needs for queries like q over this cache."""
    desc = _cache_like(k_cache, block_table)
    with torch.cuda.device(k_cache.device):
        return int(_abi.load().jvp_attn_chunk_workspace_size(desc, q.shape[1], _DT[q.dtype],
                                                             q.shape[0]))


# ---- norms of queries and keys per head, and rotation by position
def rope_table(num_positions: int, dim: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """Angles for ``norm_rope`` and ``cache_append``: float32 [num_positions, dim].

    Row p holds the cosines, then the sines, of p * base**(-2 i / dim), i < dim / 2,
    computed in 64 bits.  Any other table of this layout will do (scaled
    frequencies, positions with several axes).
    """
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and positive, got {dim}")
    i = torch.arange(dim // 2, dtype=torch.float64, device=device)
    p = torch.arange(num_positions, dtype=torch.float64, device=device)
    a = p[:, None] * torch.exp(i * (-2.0 * math.log(base) / dim))
    return torch.cat((a.cos(), a.sin()), 1).float()


def _check_rope(rope, q_weight, k_weight, D, device):
    if rope is None and q_weight is None and k_weight is None:
        raise ValueError("neither rope nor norm weights are given")
    if rope is not None:
        if (rope.dim() != 2 or rope.dtype != torch.float32 or rope.device != device
                or not rope.is_contiguous()):
            raise ValueError(f"rope must be a contiguous float32 [positions, dim] tensor on {device}")
        if rope.shape[1] % 2 or not 0 < rope.shape[1] <= D:
            raise ValueError(f"rope must have an even number of columns of at most {D}, got "
                             f"{rope.shape[1]}")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if q_weight is not None:
        for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if tuple(t.shape) != (D,) or t.device != device or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous [{D}] tensor on {device}")
            if t.dtype not in _DT or t.dtype != q_weight.dtype:
                raise TypeError("q_weight and k_weight must be float32, float16 or bfloat16, both alike")


def _check_norm_rope(q, k, dq, dk, rope, positions, q_weight, k_weight, cotangents=()):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, H, N, D]")
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if q.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    B, _, N, D = q.shape
    if k.shape[0] != B or k.shape[2] != N or k.shape[3] != D:
        raise ValueError(f"k must be [{B}, heads, {N}, {D}], got {tuple(k.shape)}")
    if (dq is None) != (dk is None):
        raise ValueError("dq and dk go together")
    named = [("q", q, q), ("k", k, k)]
    if dq is not None:
        named += [("dq", dq, q), ("dk", dk, k)]
    named += list(cotangents)
    for n, t, like in named:
        if t is None or t.shape != like.shape or t.dtype != q.dtype or t.device != q.device:
            raise ValueError(f"{n} must be a {q.dtype} tensor {tuple(like.shape)} on {q.device}")
        if t.stride(3) != 1 and t.numel() > 0 and D > 1:
            raise ValueError(f"{n} must have a unit innermost stride")
    _check_rope(rope, q_weight, k_weight, D, q.device)
    if positions is not None:
        if positions.dim() == 1:
            raise ValueError(f"positions must be [{B}, {N}] (expand those that are shared)")
        _check_int32(positions, "positions", (B, N), q.device)


def _positions(positions, q):
    """[N] as [B, N]."""
    if positions is not None and positions.dim() == 1 and q.dim() == 4:
        return positions.expand(q.shape[0], -1)
    return positions


def _rope_call(dq_dk, q, k, rope, positions, q_weight, k_weight, eps, interleaved):
    bind, entry = _native("jvp_attn_norm_rope")
    layout = (q, k, *dq_dk, rope, _positions(positions, q), q_weight, k_weight)
    r = bind.rope(entry, *layout, eps, interleaved)
    if r is None:  # a layout not seen before
        _check_norm_rope(*layout)
        bind.remember(bind.ROPE, 0, *layout)
        r = bind.rope(entry, *layout, eps, interleaved)
    if type(r) is int:
        _abi.check(r)
    return r


def _rope_bwd_call(tensors, g, rope, positions, q_weight, k_weight, eps, interleaved):
    bind, entry = _native("jvp_attn_norm_rope_bwd")
    rest = (rope, _positions(positions, tensors[0]), q_weight, k_weight)
    r = bind.rope_bwd(entry, *tensors, *g, *rest, eps, interleaved)
    if r is None:  # a layout not seen before
        q, k, dq, _ = tensors
        names = (("g_q", g[0], q), ("g_k", g[1], k), ("g_dq", g[2], q), ("g_dk", g[3], k))
        _check_norm_rope(*tensors, *rest, cotangents=names if dq is not None else names[:2])
        with torch.cuda.device(q.device):
            need = int(_abi.load().jvp_attn_norm_rope_bwd_workspace_size(q.shape[3]))
        bind.remember(bind.ROPE_BWD, need, *tensors, *g, *rest)
        r = bind.rope_bwd(entry, *tensors, *g, *rest, eps, interleaved)
    if type(r) is int:
        _abi.check(r)
    return r


def norm_rope(q: torch.Tensor, k: torch.Tensor, rope: Optional[torch.Tensor] = None,
              positions: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
              k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
              interleaved: bool = False):
    """Queries [B, H, N, D] and keys [B, Hkv, N, D] normalised per head and rotated by position.

    Per row: x * rsqrt(mean(x**2) + eps) * weight over the head dimension (without
    weights no norm), then the first ``rope.shape[1]`` columns rotated in pairs by the
    angles of the row's position: ``rope`` is float32 [positions, dim], cosines then
    sines (``rope_table``; None: no rotation); pairs are columns (i, i + dim / 2), or
    (2 i, 2 i + 1) with ``interleaved``.  ``positions`` (int32 [N] or [B, N], on the
    device) defaults to 0 .. N - 1; one that is no row of the table is reported by
    ``device_status`` (JVP_ERR_INDEX), and the outputs' rows of its token are not
    written.  Computed in float32; returns (q, k) in q's dtype.  ``autograd.norm_rope``
    is the differentiable form.
    """
    return _rope_call((None, None), q, k, rope, positions, q_weight, k_weight, eps, interleaved)


def norm_rope_dual(q: torch.Tensor, k: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                   rope: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                   q_weight: Optional[torch.Tensor] = None,
                   k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   interleaved: bool = False):
    """``norm_rope`` with tangents dq, dk of q and k: (q, k, dq, dk) from one pass."""
    return _rope_call((dq, dk), q, k, rope, positions, q_weight, k_weight, eps, interleaved)


def norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, g_q: torch.Tensor, g_k: torch.Tensor,
                  rope: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                  q_weight: Optional[torch.Tensor] = None,
                  k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  interleaved: bool = False):
    """Gradients (q, k, q_weight, k_weight) of ``norm_rope`` for cotangents g_q, g_k.

    Those of the weights are float32 (None without norms), summed in a fixed order.
    """
    return _rope_bwd_call((q, k, None, None), (g_q, g_k, None, None), rope, positions, q_weight,
                          k_weight, eps, interleaved)


def norm_rope_bwd_dual(q: torch.Tensor, k: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                       g_q: torch.Tensor, g_k: torch.Tensor, g_dq: torch.Tensor,
                       g_dk: torch.Tensor, rope: Optional[torch.Tensor] = None,
                       positions: Optional[torch.Tensor] = None,
                       q_weight: Optional[torch.Tensor] = None,
                       k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       interleaved: bool = False):
    """Gradients (q, k, dq, dk, q_weight, k_weight) of ``norm_rope_dual``."""
    return _rope_bwd_call((q, k, dq, dk), (g_q, g_k, g_dq, g_dk), rope, positions, q_weight,
                          k_weight, eps, interleaved)


def _check_append(q, k, v, k_cache, v_cache, block_table, rope, start_pos, cu_seqlens, q_weight,
                  k_weight, k_scale, v_scale, out):
    _check_rows(k, v, k_cache, v_cache, block_table, start_pos, cu_seqlens, k_scale, v_scale)
    T, D, dev = k.shape[0], k_cache.shape[3], k_cache.device
    H = q.shape[1] if q.dim() == 3 else -1
    _check_packed(q, "q", k.dtype, dev, (T, H, D))
    if out is not None:
        _check_packed(out, "out", k.dtype, dev, (T, H, D))
    _check_rope(rope, q_weight, k_weight, D, dev)


def cache_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, block_table: torch.Tensor,
                 rope: Optional[torch.Tensor] = None, start_pos: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None,
                 q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """``cache_write`` of keys that are normalised and rotated on the way, with the queries.

    q is [T, H, D], k and v [T, Hkv, D]: the new rows as they leave their projections.
    A row's position in its sequence (``start_pos[b]`` + its place among the sequence's
    rows) is its row of ``rope``; rope, weights, eps and interleaved are those of
    ``norm_rope``, and the rest of the arguments those of ``cache_write``.  Returns the
    normalised and rotated queries [T, H, D] (``out`` if given; it may be q itself),
    for ``attention_chunk`` or ``attention_decode``.  The cache holds what ``norm_rope``
    and ``cache_write`` would leave there.  Tokens whose place is out of range, or
    whose position is no row of rope, are skipped whole and reported by
    ``device_status`` (JVP_ERR_INDEX); rows that belong to no sequence are ignored.
    """
    bind, entry = _native("jvp_attn_cache_append")
    layout = (q, k, v, k_cache, v_cache, block_table, rope, start_pos, cu_seqlens, q_weight,
              k_weight, k_scale, v_scale, out)
    r = bind.append(entry, *layout, eps, interleaved)
    if r is None:  # a layout not seen before
        _check_append(*layout)
        bind.remember(bind.APPEND, 0, *layout)
        r = bind.append(entry, *layout, eps, interleaved)
    if type(r) is int:
        _abi.check(r)
    return r


def device_status(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise the stream and return (and clear) the library's device status."""
    lib = _abi.load()
    s = (stream or torch.cuda.current_stream()).cuda_stream
    return int(lib.jvp_attn_get_device_status(ctypes.c_void_p(s)))


def last_path() -> int:
    """Kernel family of the last call on this thread: 1 tensor-core, 2 CUDA-core,
    3 tensor-core with split-KV and the merge kernel, 4 tensor-core with each
    query tile's key range split between the two CTAs of a cluster."""
    return int(_abi.load().jvp_attn_debug_last_path())


TENSOR_CORE_PATHS = (1, 3, 4)


def set_cluster_split(enable: bool) -> None:
    """Diagnostic: allow (default) or forbid the cluster key split (process-wide)."""
    _abi.check(_abi.load().jvp_attn_debug_set_cluster_split(1 if enable else 0))
