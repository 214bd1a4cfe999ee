"""Refusals of the packed-prompt and paged-cache entry points: every one before
a device is touched."""

import ctypes

import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build

P = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def cache(pages=8, page=16, Hkv=2, D=64, B=3, max_pages=4, stride=None, dtype=_abi.JVP_BF16,
          ks=None, vs=None):
    full = _abi.Strides(Hkv * page * D, page * D, D, 1)
    return _abi.Cache(pages, page, Hkv, D, B, max_pages, max_pages if stride is None else stride,
                      dtype, ks or full, vs or full)


def rows(n=2, Hkv=2, D=64, d=1):
    return (_abi.Strides * 2)(*[_abi.Strides(0, D, Hkv * D, d)] * n)


def write(lib, c=None, dtype=_abi.JVP_BF16, T=3, k=P, strides=None, table=P, cu=None, kc=P, sc=P,
          no_cache=False):
    return lib.jvp_attn_cache_write(None if no_cache else ctypes.byref(c or cache()), dtype, T, k, k,
                                    rows() if strides is None else strides, table, None, cu, kc, kc,
                                    sc, sc, None)


def read(lib, c=None, dtype=_abi.JVP_BF16, T=3, k=P, strides=None, table=P, cu=None, kc=P, sc=P):
    return lib.jvp_attn_cache_read(ctypes.byref(c or cache()), dtype, T, kc, kc, sc, sc, table, None,
                                   cu, k, k, rows() if strides is None else strides, None)


def decode(lib, c=None, H=4, dtype=_abi.JVP_BF16, q=P, qs=None, table=P, lens=P, scale=0.125, o=P,
           os=None, kc=P, sc=P, lse=None):
    st = _abi.Strides(H * 64, 64, 0, 1)
    return lib.jvp_attn_decode(ctypes.byref(c or cache()), H, dtype, q, qs or st, kc, kc, sc, sc,
                               table, lens, scale, o, os or st, lse, P, 1 << 30, None)


@pytest.mark.parametrize("call", [write, read, decode])
def test_cache_descriptions(lib, call):
    BAD, UNS = _abi.JVP_ERR_INVALID_ARG, _abi.JVP_ERR_UNSUPPORTED
    assert call(lib, cache(D=0)) == BAD
    assert call(lib, cache(D=129)) == UNS
    assert call(lib, cache(page=0)) == BAD
    assert call(lib, cache(pages=-1)) == BAD
    assert call(lib, cache(max_pages=-1)) == BAD
    assert call(lib, cache(stride=3)) == BAD                      # rows of the table overlap
    assert call(lib, cache(dtype=9)) == BAD
    assert call(lib, cache(dtype=_abi.JVP_F16)) == BAD            # neither bf16 nor e4m3
    assert call(lib, cache(pages=1 << 31)) == UNS
    assert call(lib, cache(page=1 << 16, max_pages=1 << 15)) == UNS
    assert call(lib, cache(page=(1 << 31) - 1023, max_pages=1)) == UNS  # a tile's end past 2^31
    assert call(lib, cache(page=1, max_pages=(1 << 31) - 1, stride=1 << 31)) == UNS
    assert call(lib, cache(ks=_abi.Strides(2048, 1024, 64, 2))) == BAD
    assert call(lib, cache(vs=_abi.Strides(2048, -1024, 64, 1))) == BAD
    assert call(lib, kc=None) == BAD
    assert call(lib, kc=ctypes.c_void_p(0x10001)) == _abi.JVP_ERR_ALIGNMENT
    assert call(lib, cache(dtype=_abi.JVP_E4M3), sc=None) == BAD  # scales are needed
    assert call(lib, table=None) == BAD
    assert call(lib, table=ctypes.c_void_p(0x10002)) == _abi.JVP_ERR_ALIGNMENT
    assert call(lib, dtype=_abi.JVP_E4M3) == BAD                  # rows and queries are not e4m3
    assert lib.jvp_attn_debug_last_path() == 0


def test_rows(lib):
    BAD = _abi.JVP_ERR_INVALID_ARG
    for call in (write, read):
        assert call(lib, T=-1) == BAD
        assert call(lib, T=2) == BAD                               # without cu_seqlens: T = B
        assert call(lib, T=1 << 31, cu=P) == _abi.JVP_ERR_UNSUPPORTED
        assert call(lib, k=None) == BAD
        assert call(lib, k=ctypes.c_void_p(0x10001)) == _abi.JVP_ERR_ALIGNMENT
        assert call(lib, strides=rows(d=2)) == BAD
        assert call(lib, T=0, cu=P, k=None, kc=None, table=None) == _abi.JVP_OK
        assert call(lib, cache(B=0), T=0, k=None, kc=None, table=None) == _abi.JVP_OK
    flat = (_abi.Strides * 2)(*[_abi.Strides(0, 64, 0, 1)] * 2)
    assert read(lib, strides=flat) == BAD                          # outputs on top of each other
    assert write(lib, cache(ks=_abi.Strides(0, 1024, 64, 1))) == BAD
    assert write(lib, no_cache=True) == BAD
    assert b"NULL" in lib.jvp_attn_last_error()


def test_decode(lib):
    BAD = _abi.JVP_ERR_INVALID_ARG
    assert decode(lib, H=3) == BAD
    assert b"multiple of Hkv" in lib.jvp_attn_last_error()
    assert decode(lib, H=-2) == BAD
    assert decode(lib, cache(B=1 << 20), H=1 << 20) == _abi.JVP_ERR_UNSUPPORTED
    assert decode(lib, scale=float("nan")) == BAD
    assert decode(lib, q=None) == BAD and decode(lib, o=None) == BAD and decode(lib, lens=None) == BAD
    assert decode(lib, lse=ctypes.c_void_p(0x10002)) == _abi.JVP_ERR_ALIGNMENT
    assert decode(lib, os=_abi.Strides(0, 64, 0, 1)) == BAD
    assert decode(lib, qs=_abi.Strides(256, 64, 0, 2)) == BAD
    assert decode(lib, cache(B=0), q=None, o=None, lens=None) == _abi.JVP_OK
    assert lib.jvp_attn_decode_workspace_size(None, 4, _abi.JVP_BF16) == 0
    assert lib.jvp_attn_decode_workspace_size(cache(), 3, _abi.JVP_BF16) == 0
    assert lib.jvp_attn_decode_workspace_size(cache(), 4, _abi.JVP_BF16) == 0  # no device here


def test_status_of_a_bad_index_has_a_name(lib):
    assert b"out of range" in lib.jvp_attn_status_string(_abi.JVP_ERR_INDEX)


def test_the_binding_refuses_before_it_calls():
    """Shapes, types and devices that the Python functions check themselves."""
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    x, q = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for bad in (lambda: api.cache_write(x, x, c, c, t, n), lambda: api.cache_read(c, c, t, n),
                lambda: api.attention_decode(q, c, c, t, n)):
        with pytest.raises(ValueError, match="CUDA"):
            bad()
    with pytest.raises(ValueError, match="num_rows"):
        api.cache_read(c, c, t, n, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="pages"):
        api.cache_write(x, x, c[0], c[0], t, n)
    with pytest.raises(TypeError):
        api.attention_decode(q, c.long(), c.long(), t, n)


def packed(lib, T=8, B=2, H=4, Hkv=2, D=64, dtype=_abi.JVP_BF16, ptr=P, cu=P, causal=1, scale=0.125,
           ins=None, outs=None, lse=None, no_shape=False):
    sh = _abi.PackedShape(T, B, H, Hkv, D)
    st = _abi.Strides(0, 64, 256, 1)
    return lib.jvp_attn_fwd_packed(None if no_shape else ctypes.byref(sh), dtype, ptr, ptr, ptr,
                                   ins or (_abi.Strides * 3)(st, st, st), cu, causal, scale, ptr,
                                   outs or st, lse, None)


def test_packed(lib):
    BAD, UNS = _abi.JVP_ERR_INVALID_ARG, _abi.JVP_ERR_UNSUPPORTED
    assert packed(lib, no_shape=True) == BAD
    for kw in (dict(T=-1), dict(B=-1), dict(H=-1), dict(Hkv=-1), dict(D=0), dict(Hkv=3),
               dict(dtype=_abi.JVP_E4M3), dict(dtype=7), dict(causal=2), dict(scale=float("inf")),
               dict(ptr=None), dict(cu=None), dict(outs=_abi.Strides(0, 64, 0, 1)),
               dict(outs=_abi.Strides(0, 0, 256, 1)), dict(outs=_abi.Strides(0, 64, -256, 1)),
               dict(ins=(_abi.Strides * 3)(*[_abi.Strides(0, 64, 256, 2)] * 3))):
        assert packed(lib, **kw) == BAD, kw
    for kw in (dict(D=136), dict(T=1 << 31), dict(B=1 << 31), dict(T=1 << 30, H=4),
               dict(T=(1 << 31) - 1024, B=1, H=1, Hkv=1), dict(T=8, B=(1 << 31) - 1031, H=1, Hkv=1)):
        assert packed(lib, **kw) == UNS, kw
    for kw in (dict(ptr=ctypes.c_void_p(0x10001)), dict(cu=ctypes.c_void_p(0x10002)),
               dict(lse=ctypes.c_void_p(0x10002))):
        assert packed(lib, **kw) == _abi.JVP_ERR_ALIGNMENT, kw
    for kw in (dict(T=0), dict(B=0), dict(H=0, Hkv=0)):
        assert packed(lib, ptr=None, cu=None, **kw) == _abi.JVP_OK, kw
    assert lib.jvp_attn_debug_last_path() == 0


def test_the_packed_binding_refuses_before_it_calls():
    q, k = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.attention_packed(q, k, k, cu)
    with pytest.raises(ValueError, match="T, H, D"):
        api.attention_packed(q[0], k, k, cu)
    with pytest.raises(TypeError):
        api.attention_packed(q.long(), k.long(), k.long(), cu)
