"""Refusals of the norms and rotation of queries and keys, without a GPU."""

import ctypes

import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build

P = 0x10000  # an address that is never followed
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def rope(table=P, rows=64, dim=64, interleaved=0, wdt=0, qw=P, kw=P, eps=1e-6):
    return _abi.Rope(table, rows, dim, interleaved, wdt, qw, kw, eps)


def strides(records, **first):
    s = (_abi.Strides * records)(*[_abi.Strides(4096, 1024, 64, 1) for _ in range(records)])
    for name, value in first.items():
        setattr(s[0], name, value)
    return s


def dense(lib, r=None, shape=(1, 2, 16, 16, 64, 1), dtype=2, positions=None, pstride=0, q=P, tan=None,
          ins=None, outs=None, y=P):
    return lib.jvp_attn_norm_rope(
        ctypes.byref(_abi.Shape(*shape)) if shape else None, dtype,
        ctypes.byref(r if r is not None else rope()), positions, pstride, q, P, tan, tan,
        ins if ins is not None else strides(4), y, P, tan, tan,
        outs if outs is not None else strides(4), None)


def bwd(lib, r=None, g=P, gw=P, ws=P, bytes_=0, ins=None):
    return lib.jvp_attn_norm_rope_bwd(
        ctypes.byref(_abi.Shape(1, 2, 16, 16, 64, 1)), 2, ctypes.byref(r if r is not None else rope()),
        None, 0, P, P, None, None, g, P, None, None, ins if ins is not None else strides(8), P, P, None,
        None, strides(4), gw, gw, ws, bytes_, None)


def cache(dtype=2, pages=8, page=16, Hkv=2, D=64, B=3, cols=4):
    s = _abi.Strides(Hkv * page * D, page * D, D, 1)
    return _abi.Cache(pages, page, Hkv, D, B, cols, cols, dtype, s, s)


def append(lib, c=None, r=None, H=4, dtype=2, T=3, q=P, cu=P, ins=None, out=P, outs=None, ks=None):
    return lib.jvp_attn_cache_append(
        ctypes.byref(c if c is not None else cache()), H, dtype, T, q, P, P,
        ins if ins is not None else strides(3), ctypes.byref(r if r is not None else rope()), P, P, cu,
        out, outs if outs is not None else strides(1), P, P, ks, ks, None)


INVALID, UNSUPPORTED, ALIGNMENT = (_abi.JVP_ERR_INVALID_ARG, _abi.JVP_ERR_UNSUPPORTED,
                                   _abi.JVP_ERR_ALIGNMENT)


@pytest.mark.parametrize("call", [dense, bwd, lambda lib, r: append(lib, r=r)])
def test_angles_and_weights(lib, call):
    for r, want in ((rope(dim=65), INVALID), (rope(dim=66), INVALID), (rope(dim=-2), INVALID),
                    (rope(rows=-1), INVALID), (rope(rows=BIG), UNSUPPORTED), (rope(table=None), INVALID),
                    (rope(table=P + 2), ALIGNMENT), (rope(interleaved=2), INVALID),
                    (rope(kw=None), INVALID), (rope(qw=None), INVALID), (rope(wdt=3), INVALID),
                    (rope(qw=P + 2), ALIGNMENT), (rope(dim=0, qw=None, kw=None), INVALID),
                    (rope(eps=-1.0), INVALID), (rope(eps=float("nan")), INVALID),
                    (rope(eps=float("inf")), INVALID)):
        assert call(lib, r) == want, lib.jvp_attn_last_error()


def test_dense_rows(lib):
    assert dense(lib, shape=None) == INVALID
    assert dense(lib, shape=(1, 2, 16, 17, 64, 1)) == INVALID
    assert dense(lib, shape=(-1, 2, 16, 16, 64, 1)) == INVALID
    assert dense(lib, shape=(1, 2, 16, 16, 0, 1)) == INVALID
    assert dense(lib, shape=(1, 2, 16, 16, 129, 1)) == UNSUPPORTED
    assert dense(lib, rope(rows=BIG - 1), shape=(1 << 20, 2, 1 << 12, 1 << 12, 64, 1)) == UNSUPPORTED
    assert dense(lib, rope(rows=15)) == INVALID  # fewer rows than tokens
    assert dense(lib, dtype=3) == INVALID
    assert dense(lib, q=None) == INVALID and dense(lib, y=None) == INVALID
    assert dense(lib, q=P + 1) == ALIGNMENT and dense(lib, y=P + 1) == ALIGNMENT
    assert dense(lib, positions=P + 2) == ALIGNMENT
    assert dense(lib, positions=P, pstride=-1) == INVALID
    assert dense(lib, ins=strides(4, d=2)) == INVALID and dense(lib, ins=strides(4, n=-1)) == INVALID
    assert dense(lib, outs=strides(4, h=0)) == INVALID
    assert dense(lib, shape=(0, 2, 16, 16, 64, 1), q=None) == _abi.JVP_OK
    assert bwd(lib, g=None) == INVALID and bwd(lib, gw=None) == INVALID
    assert bwd(lib, ws=P + 2) == ALIGNMENT and bwd(lib, gw=P + 2) == ALIGNMENT
    assert lib.jvp_attn_norm_rope_bwd_workspace_size(0) == 0
    assert lib.jvp_attn_norm_rope_bwd_workspace_size(129) == 0


def test_rows_into_the_cache(lib):
    assert append(lib, H=-1) == INVALID and append(lib, T=-1) == INVALID
    assert append(lib, T=BIG) == UNSUPPORTED and append(lib, H=BIG) == UNSUPPORTED
    assert append(lib, dtype=0) == INVALID and append(lib, dtype=3) == INVALID
    assert append(lib, cache(dtype=3)) == INVALID  # no scales
    assert append(lib, T=4, cu=None) == INVALID
    assert append(lib, q=None) == INVALID and append(lib, out=None) == INVALID
    assert append(lib, out=P + 1) == ALIGNMENT and append(lib, cu=P + 2) == ALIGNMENT
    assert append(lib, ins=strides(3, d=0)) == INVALID and append(lib, outs=strides(1, h=0)) == INVALID
    assert append(lib, cache(D=129)) == UNSUPPORTED
    assert append(lib, T=0, q=None, out=None) == _abi.JVP_OK


def test_the_binding_refuses(lib):
    q = torch.zeros(1, 2, 3, 8)
    for call in (lambda: api.norm_rope(q, q), lambda: api.norm_rope_dual(q, q, q, q),
                 lambda: api.norm_rope_bwd(q, q, q, q), lambda: api.norm_rope(q[0], q)):
        with pytest.raises(ValueError):
            call()
    c, t = torch.zeros(2, 2, 4, 8), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.cache_append(q[0], q[0], q[0], c, c, t)
    for dim in (0, 7, -2):
        with pytest.raises(ValueError):
            api.rope_table(4, dim)


def test_angles_of_far_positions():
    """Rounded once from 64 bits: half a unit of fp32 at 1, and the 64-bit angle's own error
    (position 2^-53 times a few)."""
    import math
    t = api.rope_table(1 << 16, 64)
    for p in (0, 1, 12345, (1 << 16) - 1):
        for i in (0, 1, 15, 31):
            a = p * 10000.0 ** (-2 * i / 64)
            assert abs(t[p, i].item() - math.cos(a)) <= 2.0 ** -24 + p * 2.0 ** -50
            assert abs(t[p, 32 + i].item() - math.sin(a)) <= 2.0 ** -24 + p * 2.0 ** -50
