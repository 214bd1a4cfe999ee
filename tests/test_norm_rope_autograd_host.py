"""How autograd.norm_rope wires its kernels into autograd, without a GPU."""

import pytest
import rope_autograd as ra
import torch
from forward_mode_flash_gb300 import api

TABLE = api.rope_table(ra.N, 8)


@pytest.fixture(autouse=True)
def kernels(monkeypatch):
    ra.plain_kernels(monkeypatch)


some = pytest.mark.parametrize("which", ra.SOME, ids=lambda w: "-".join(ra.NAMES[i] for i in w))
ways = pytest.mark.parametrize("way", [ra.train_through_jvp, ra.train_through_dual_tensors],
                               ids=lambda f: f.__name__)


@some
@ways
def test_tangents_of_some_arguments(way, which):
    ra.compare(way, lambda x: x, TABLE, which)
