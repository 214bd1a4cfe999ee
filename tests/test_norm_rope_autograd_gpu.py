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


@some
@pytest.mark.parametrize("way", [ra.gradients, ra.pulled_back], ids=lambda f: f.__name__)
def test_transforms_of_torch_func(way, which):
    ra.compare(way, cuda, TABLE, which)


@some
def test_gradients_of_tangents(which):
    ra.compare(ra.grad_of_jvp, cuda, TABLE, which)
    if len(which) < 4:
        ra.compare(ra.grad_of_others, cuda, TABLE, which)


def test_gradients_of_gradients_are_refused():
    """Also where the cotangents are constants, and within torch.func."""
    c, table = [x.cuda() for x in ra.data()[2]], TABLE.cuda()
    args = [x.cuda().requires_grad_() for x in ra.data()[0]]
    y = ra.own(table)(*args)
    g = torch.autograd.grad(ra.loss(y, (), c), args[0], create_graph=True)[0]
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((g ** 2).sum() + args[0].sum()).backward()

    def first(q):
        return torch.func.grad(lambda q: ra.loss(ra.own(table)(q, *args[1:]), (), c))(q).sum()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        torch.func.grad(first)(args[0].detach())


@some
@pytest.mark.parametrize("way", [ra.tangents_of_gradients, ra.tangents_of_gradients_by_dual_tensors],
                         ids=lambda f: f.__name__)
def test_tangents_of_gradients(way, which):
    ra.compare(way, cuda, TABLE, which)


def test_what_has_no_derivative_is_refused():
    """Tangents of tangents, and of the gradients of tangents."""
    args, tangents, c = ([x.cuda() for x in z] for z in ra.data())
    f = ra.own(TABLE.cuda())

    def tangent(q):
        return torch.func.jvp(lambda q: f(q, *args[1:]), (q,), (tangents[0],))[1]
    with pytest.raises(RuntimeError, match="tangents of tangents"):
        torch.func.jvp(tangent, (args[0],), (tangents[0],))

    with ra.fwAD.dual_level():
        y = f(ra.fwAD.make_dual(args[0].requires_grad_(), tangents[0]), *args[1:])
        t = ra.fwAD.unpack_dual(y[0]).tangent
        with pytest.raises(RuntimeError, match="gradients of tangents"):
            t.sum().backward()


@some
@pytest.mark.parametrize("way", [ra.train_through_jvp, ra.values_by_dual_tensors],
                         ids=lambda f: f.__name__)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_one_rounding_of_the_result(dtype, way, which):
    """In 16 bits, also where the tangents are sums of those by the rows and the weights."""
    ra.compare(way, cuda, TABLE, which, dtype=dtype)
