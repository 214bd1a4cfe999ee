"""The native part of the binding, without a GPU: it calls nothing for layouts it does not know,
and what it refuses becomes a Python exception."""

import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build


@pytest.fixture(scope="module")
def bind():
    build.build()
    return _abi.load_bind()


def test_the_module_is_built_for_this_pytorch(bind):
    assert torch.__version__ in build.bind_path()
    assert len({bind.PACKED, bind.WRITE, bind.READ, bind.DECODE}) == 4


def test_unknown_layouts_are_not_called(bind):
    q, cu = torch.zeros(3, 2, 8), torch.zeros(2, dtype=torch.int32)
    assert bind.packed(0, q, q, q, cu, None, False, None, True) is None
    assert bind.write(0, q, q, q, q, cu, None, None, None, None) is None
    assert bind.read(0, q, q, q, q, cu, None, None, None, None) is None
    assert bind.decode(0, q, q, q, cu, cu, None, None, None, None, None, True) is None


def test_arguments_that_are_not_tensors_are_refused(bind):
    q, cu = torch.zeros(3, 2, 8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: bind.packed(0, q, q, "k", cu, None, False, None, True),
                 lambda: bind.packed(0, q), lambda: bind.remember(),
                 lambda: bind.remember("op", 0, q), lambda: bind.empty_rows(q, 4, None),
                 lambda: bind.empty_rows(torch.zeros(1, 2, 3, 4), 4, "f32"),
                 lambda: bind.decode(0, q, 3, q, cu, cu, None, None, None, None, None, True)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(TypeError):
        api.attention_packed(q, q, [1.0], cu)


def test_a_known_layout_needs_an_entry_point(bind):
    q, cu = torch.zeros(3, 2, 24), torch.zeros(2, dtype=torch.int32)
    bind.remember(bind.PACKED, 0, q, q, q, cu, None)
    with pytest.raises(ValueError):
        bind.packed(0, q, q, q, cu, None, False, None, True)


def test_new_rows_have_the_type_of_the_cache(bind):
    for dt, want in ((torch.float16, torch.float16), (torch.float8_e4m3fn, torch.bfloat16)):
        for dtype in (None, torch.float32):
            k, v = bind.empty_rows(torch.zeros(3, 2, 8, 16).to(dt), 5, dtype)
            assert k.shape == v.shape == (5, 2, 16) and k.dtype == v.dtype == (dtype or want)
            assert k.data_ptr() != v.data_ptr()
