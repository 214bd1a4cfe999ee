"""Refusals of the attention of chunks and of the window of single tokens, without a GPU."""

import ctypes

import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build

P = 0x10000  # an address that is never followed
BAD, UNS, ALN = _abi.JVP_ERR_INVALID_ARG, _abi.JVP_ERR_UNSUPPORTED, _abi.JVP_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def cache(pages=8, page=16, Hkv=2, D=64, B=3, max_pages=4, stride=None, dtype=_abi.JVP_BF16):
    full = _abi.Strides(Hkv * page * D, page * D, D, 1)
    return _abi.Cache(pages, page, Hkv, D, B, max_pages, max_pages if stride is None else stride,
                      dtype, full, full)


def rows(H=4, D=64, n=None, d=1, h=None):
    n = H * D if n is None else n
    return _abi.Strides(n, D if h is None else h, n, d)  # (sequences of one token: b)


def chunk(lib, c=None, H=4, dtype=_abi.JVP_BF16, T=5, q=P, qs=None, kc=P, sc=None, table=P, lens=P, cu=P,
          window=0, sinks=0, scale=0.125, o=P, os=None, lse=None, no_cache=False, no_strides=False):
    return lib.jvp_attn_chunk(None if no_cache else ctypes.byref(c or cache()), H, dtype, T, q,
                              None if no_strides else qs or rows(), kc, kc, sc, sc, table, lens, cu,
                              window, sinks, scale, o, os or rows(), lse, P, 1 << 30, None)


def window(lib, c=None, H=4, dtype=_abi.JVP_BF16, q=P, qs=None, kc=P, sc=None, table=P, lens=P, window=8,
           sinks=1, scale=0.125, o=P, os=None, lse=None, no_cache=False, no_strides=False):
    return lib.jvp_attn_decode_window(None if no_cache else ctypes.byref(c or cache()), H, dtype, q,
                                      None if no_strides else qs or rows(), kc, kc, sc, sc, table, lens,
                                      window, sinks, scale, o, os or rows(), lse, P, 1 << 30, None)


@pytest.mark.parametrize("call", [chunk, window])
def test_what_both_refuse(lib, call):
    assert call(lib, no_cache=True) == BAD and call(lib, no_strides=True) == BAD
    assert call(lib, cache(D=0)) == BAD and call(lib, cache(D=129)) == UNS
    assert call(lib, cache(page=0)) == BAD and call(lib, cache(pages=-1)) == BAD
    assert call(lib, cache(stride=3)) == BAD and call(lib, cache(dtype=9)) == BAD
    assert call(lib, cache(dtype=_abi.JVP_F16)) == BAD  # another type than the queries'
    assert call(lib, cache(dtype=_abi.JVP_E4M3)) == BAD  # without scales
    assert call(lib, dtype=7) == BAD
    assert call(lib, H=3) == BAD
    assert b"multiple of Hkv" in lib.jvp_attn_last_error()
    assert call(lib, H=-2) == BAD
    assert call(lib, scale=float("nan")) == BAD and call(lib, scale=float("inf")) == BAD
    assert call(lib, window=-1) == BAD and call(lib, sinks=-1) == BAD
    assert call(lib, qs=rows(d=2)) == BAD and call(lib, os=rows(d=0)) == BAD
    assert call(lib, qs=rows(n=-64)) == BAD
    assert call(lib, os=rows(h=0)) == BAD
    for missing in ("q", "o", "kc", "table", "lens"):
        assert call(lib, **{missing: None}) == BAD, missing
    assert call(lib, q=P + 1) == ALN and call(lib, lse=P + 2) == ALN and call(lib, lens=P + 2) == ALN
    assert call(lib, cache(B=0), q=None, o=None, lens=None, kc=None, table=None) == _abi.JVP_OK
    assert call(lib, cache(Hkv=0), H=0, q=None, o=None, lens=None) == _abi.JVP_OK


def test_what_chunks_refuse(lib):
    assert chunk(lib, T=-1) == BAD
    assert chunk(lib, os=rows(n=0)) == BAD
    assert chunk(lib, cu=None) == BAD and chunk(lib, cu=P + 2) == ALN
    assert chunk(lib, T=1 << 31) == UNS and chunk(lib, T=1 << 29, H=64) == UNS
    assert chunk(lib, T=0, q=None, o=None, cu=None, lens=None) == _abi.JVP_OK
    size = lib.jvp_attn_chunk_workspace_size
    assert size(None, 4, _abi.JVP_BF16, 5) == 0 and size(cache(), 3, _abi.JVP_BF16, 5) == 0
    assert size(cache(), 4, _abi.JVP_BF16, -5) == 0
    assert size(cache(), 4, _abi.JVP_BF16, 5) == 0  # no device here


def test_the_bindings_refuse_before_they_call():
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q, cu = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for bad in (lambda: api.attention_chunk(q, c, c, t, n, cu),
                lambda: api.attention_decode(q, c, c, t, n, window=4)):
        with pytest.raises(ValueError, match="CUDA"):
            bad()
    for kw in (dict(window=0), dict(window=-1), dict(window=4, sinks=-1)):
        with pytest.raises(ValueError):
            api.attention_chunk(q, c, c, t, n, cu, **kw)
        with pytest.raises(ValueError):
            api.attention_decode(q, c, c, t, n, **kw)
    with pytest.raises(TypeError):
        api.attention_chunk(q, c.long(), c.long(), t, n, cu)
    with pytest.raises(ValueError, match="workspace"):
        api.attention_chunk(q, c, c, t, n, cu, workspace=torch.zeros(9, 2, dtype=torch.uint8)[:, 0])


@pytest.mark.parametrize("entry", ["rope", "rope_bwd", "append", "decode_window", "chunk"])
def test_the_module_refuses_what_are_no_tensors(entry):
    build.build()
    bind, _ = api._native("jvp_attn_chunk")
    with pytest.raises(TypeError):
        getattr(bind, entry)(0, 3)
    with pytest.raises(TypeError):
        getattr(bind, entry)()
