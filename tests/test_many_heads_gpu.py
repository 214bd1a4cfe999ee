"""Norms and rotation of tokens with millions of heads: work is divided by heads alone."""

import pytest
import torch
from forward_mode_flash_gb300 import _abi, api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("D", [8, 7])
@pytest.mark.parametrize("tokens,heads", [(1, (1 << 22) + 3), (3, 100003), (1, 999)])
def test_heads_as_tokens(tokens, heads, D):
    """The same rows as so many tokens of one head."""
    g = torch.Generator(device="cuda").manual_seed(heads)
    q, k, gq, gk = (torch.randn(1, h, tokens, D, generator=g, device="cuda").bfloat16()
                    for h in (heads, 1, heads, 1))
    w = [1 + torch.rand(D, generator=g, device="cuda") for _ in range(2)]
    table = api.rope_table(5, 4, device="cuda")
    at = torch.tensor([[4, 0, 2][:tokens]], dtype=torch.int32, device="cuda")
    one = lambda x: x.reshape(1, 1, heads * tokens, D)  # noqa: E731
    y = api.norm_rope(q, k, table, at, *w)
    g1 = api.norm_rope_bwd(q, k, gq, gk, table, at, *w)
    z = api.norm_rope(one(q), one(q), table, at.repeat(1, heads), *w)
    g2 = api.norm_rope_bwd(one(q), one(q), one(gq), one(gq), table, at.repeat(1, heads), *w)
    assert torch.equal(one(y[0]), z[0]) and torch.equal(one(g1[0]), g2[0])
    # sums of the same terms in another order: a chain of at most n / 500 terms in a thread
    # (some 2000 warps share the rows) and of those of 700 blocks, each step 2^-24 of the
    # terms' magnitudes: |n| <= sqrt(D), a rotated pair of cotangents at most their sum
    n = heads * tokens
    mag = 2 * D ** 0.5 * one(gq).double().abs().sum((0, 1, 2)).max()
    assert (g1[2] - g2[2]).abs().max() <= 2 * (n / 500 + 700) * 2.0 ** -24 * mag
    assert api.device_status() == _abi.JVP_OK
