"""Packed prompts, the paged cache and the single-token attention on the debug
build of the library: the same bits as the ordinary build, and a clean device
status after the kernels' bounds checks."""

import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug_path():
    yield build.build(debug=True)
    _abi.use_debug_build(None)


def both(debug_path, call):
    """Results of a call on the ordinary and on the debug build."""
    out = []
    for path in (None, debug_path):
        _abi.use_debug_build(path)
        out.append([t.clone() for t in call()])
        assert api.device_status() == 0, path
    _abi.use_debug_build(None)
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[1, 130, 300, 0, 77], [1500, 1025, 1300]], ids=["short", "long"])
@pytest.mark.parametrize("dt,H,Hkv,D", [(torch.bfloat16, 8, 2, 128), (torch.float16, 4, 4, 64),
                                        (torch.float16, 3, 1, 40)])
def test_packed(debug_path, dt, H, Hkv, D, lens, causal):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(sum(lens), h, D, generator=g).to(dt).cuda() for h in (H, Hkv, Hkv))
    v[sum(lens) - 3, 0, 1] = float("inf")
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    both(debug_path, lambda: api.attention_packed(q, k, v, cu, is_causal=causal, return_lse=True))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dt,H,Hkv,D,page", [(torch.bfloat16, 8, 2, 128, 16),
                                             (torch.float16, 24, 1, 64, 24),
                                             (torch.float32, 4, 2, 96, 8)])
def test_cache_and_decode(debug_path, dt, H, Hkv, D, page, e4m3):
    lens = [1, 700, 0, 5000, 333]
    B, pages = len(lens), [-(-n // page) for n in lens]
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(sum(lens), Hkv, D, generator=g).to(dt).cuda() for _ in range(2))
    q = torch.randn(B, H, D, generator=g).to(dt).cuda()
    order = torch.randperm(sum(pages), generator=g).to(torch.int32)
    table = torch.zeros(B, max(pages), dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    table, n32 = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()

    def call():
        ct = torch.float8_e4m3fn if e4m3 else dt
        kc, vc = (torch.zeros(sum(pages), Hkv, page, D, device="cuda").to(ct) for _ in range(2))
        sc = [torch.zeros(sum(pages), Hkv, page, dtype=torch.uint8, device="cuda")
              for _ in range(2)] if e4m3 else [None, None]
        api.cache_write(k, v, kc, vc, table, cu_seqlens=cu, k_scale=sc[0], v_scale=sc[1])
        rk, rv = api.cache_read(kc, vc, table, cu_seqlens=cu, num_rows=sum(lens), k_scale=sc[0],
                                v_scale=sc[1], dtype=dt)
        o, lse = api.attention_decode(q, kc, vc, table, n32, k_scale=sc[0], v_scale=sc[1],
                                      return_lse=True)
        return rk, rv, o, lse

    both(debug_path, call)
