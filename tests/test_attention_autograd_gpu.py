"""Attention differentiated where only some arguments have tangents."""

import attention_autograd as aa
import pytest
import rope_autograd as ra
from forward_mode_flash_gb300 import api

pytestmark = pytest.mark.gpu
TABLE = api.rope_table(aa.N, 8)


def to(x):
    return x.cuda()


def name(names):
    return lambda which: "-".join(names[i] for i in which)


ways = pytest.mark.parametrize("way", [ra.train_through_jvp, ra.train_through_dual_tensors],
                               ids=lambda f: f.__name__)


@pytest.mark.parametrize("which", aa.SOME, ids=name(aa.NAMES))
@ways
def test_tangents_of_some_arguments(way, which):
    aa.compare(way, to, which)


@pytest.mark.parametrize("which", aa.MORE, ids=name(aa.MORE_NAMES))
@ways
def test_behind_norms_and_rotation(way, which):
    aa.compare(way, to, which, TABLE)
