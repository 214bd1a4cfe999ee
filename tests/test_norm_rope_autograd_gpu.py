"""autograd.norm_rope in the ways that torch differentiates, on its kernels."""

import pytest
import rope_autograd as ra
import torch
from forward_mode_flash_gb300 import api

pytestmark = pytest.mark.gpu
TABLE = api.rope_table(ra.N, 8)


def cuda(x):
    return x.cuda()


some = pytest.mark.parametrize("which", ra.SOME, ids=lambda w: "-".join(ra.NAMES[i] for i in w))
ways = pytest.mark.parametrize("way", [ra.train_through_jvp, ra.train_through_dual_tensors],
                               ids=lambda f: f.__name__)


@some
@ways
def test_tangents_of_some_arguments(way, which):
    ra.compare(way, cuda, TABLE, which)
