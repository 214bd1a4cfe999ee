"""The layouts that the binding's native part remembers, while an allocation of
its own runs Python code."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from forward_mode_flash_gb300 import _abi, build


@pytest.fixture(scope="module")
def bind():
    build.build()
    return _abi.load_bind()


def test_layouts_forgotten_during_a_call(bind):
    """Layouts enough to replace all are remembered while the output is allocated: the
    workspace still has the size of the call's own."""
    q, kc = torch.zeros(2, 4, 24), torch.zeros(3, 2, 8, 24)
    table, lens = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    layout = (q, kc, kc, table, lens, None, None, None)
    bind.remember(bind.DECODE, 123456, *layout)
    sizes = []

    class Mode(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if func is torch.ops.aten.empty.memory_format:
                if not sizes:
                    for i in range(1100):
                        bind.remember(100 + i, 1 << 40)
                sizes.append(tuple(args[0]))
            return func(*args, **(kwargs or {}))

    with Mode(), pytest.raises(RuntimeError):  # (these tensors are on no CUDA device)
        bind.decode(1, *layout, None, None, False)
    assert sizes == [(2, 4, 24), (123456,)]
    assert bind.decode(1, *layout, None, None, False) is None
