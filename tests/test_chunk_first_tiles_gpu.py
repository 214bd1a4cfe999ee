"""The first tiles of a call, which land in shared memory where each CTA worked out its part."""

import pytest
import torch
from forward_mode_flash_gb300 import _abi, api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# as many sequences as the scratch holds, more, and few; pages copied as boxes of a page, of
# codes, and row by row
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,e4m3", [(16, False), (128, False), (16, True), (12, False)])
@pytest.mark.parametrize("B,new,keys", [(2048, 1, 40), (2500, 2, 20), (300, 3, 200), (5, 700, 900)])
def test_calls_give_the_same_bits(B, new, keys, page, e4m3, D):
    """In a row on two streams, against single tokens and calls by themselves."""
    H, Hkv = 4, 1
    g = torch.Generator(device="cuda").manual_seed(B)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    cols = -(-keys // page)
    shape = (B * cols, Hkv, page, D)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v = (r(*shape).to(kind) for _ in range(2))
    scales = [torch.full(shape[:3], 125 + i, dtype=torch.uint8, device="cuda") if e4m3 else None
              for i in range(2)]
    table = torch.randperm(B * cols, generator=g, device="cuda").int().view(B, cols)
    lens = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, new * (B + 1), new, dtype=torch.int32, device="cuda")
    q = r(B * new, H, D).bfloat16()

    def call():
        return api.attention_chunk(q, k, v, table, lens, cu, k_scale=scales[0], v_scale=scales[1])

    want = call()
    assert api.last_path() == 1
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            got += [call() for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    # every sequence's last token sees all its keys.  Each output is an average of values with
    # weights within 2^-8 relatively (one rounding), rounded once more, here and there (the
    # single tokens' weights over e4m3: 2^-11)
    one = api.attention_decode(q[new - 1::new].contiguous(), k, v, table, lens, k_scale=scales[0],
                               v_scale=scales[1])
    most = v.float().abs().max() * (0.5 if e4m3 else 1.0)
    assert (want[new - 1::new].float() - one.float()).abs().max() <= 6 * 2.0 ** -8 * most
    assert api.device_status() == _abi.JVP_OK
