"""Sizes that the paged cache's entry points refuse, before a device is touched."""

import ctypes

import pytest

from forward_mode_flash_gb300 import _abi, build

P = ctypes.c_void_p(0x10000)
BF16 = _abi.JVP_BF16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def cache(pages=8, page=16, Hkv=2, D=64, B=3, max_pages=4):
    st = _abi.Strides(Hkv * page * D, page * D, D, 1)
    return ctypes.byref(_abi.Cache(pages, page, Hkv, D, B, max_pages, max_pages, BF16, st, st))


def row_calls(lib, c, T):
    """Statuses of a write and a read."""
    rows = (_abi.Strides * 2)(*[_abi.Strides(0, 64, 1 << 40, 1)] * 2)
    return [lib.jvp_attn_cache_write(c, BF16, T, P, P, rows, P, None, P, P, P, None, None, None),
            lib.jvp_attn_cache_read(c, BF16, T, P, P, None, None, P, None, P, P, P, rows, None)]


@pytest.mark.parametrize("B", [(1 << 31) - 1023, (1 << 31) - 1])
def test_numbers_of_sequences(lib, B):
    c, st = cache(B=B, Hkv=1), _abi.Strides(64, 64, 0, 1)
    calls = row_calls(lib, c, 4) + [lib.jvp_attn_decode(c, 1, BF16, P, st, P, P, None, None, P, P, 0.125,
                                                        P, st, None, P, 1 << 40, None)]
    assert calls == [_abi.JVP_ERR_UNSUPPORTED] * 3
    assert b"2^31 - 1024" in lib.jvp_attn_last_error()


def test_numbers_of_heads(lib):
    for Hkv in ((1 << 30) - 64, 1 << 30, (1 << 31) - 1):
        c = cache(Hkv=Hkv, page=1, pages=1, B=1, max_pages=1, D=1)
        assert row_calls(lib, c, 1) == [_abi.JVP_ERR_UNSUPPORTED] * 2
        assert b"Hkv" in lib.jvp_attn_last_error()
