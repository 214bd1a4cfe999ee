"""Norms and rotation, rows appended, attention of chunks and windows on the debug build of the
library: the same bits as the ordinary build, and a clean status after the kernels' bounds checks."""

import pytest
import torch

from forward_mode_flash_gb300 import api
from serving_ref import Cache
from test_serving_debug_checks_gpu import both, debug_path  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt,D,rot", [(torch.bfloat16, 128, 128), (torch.float16, 64, 32),
                                      (torch.float32, 96, 96), (torch.bfloat16, 33, 6)])
def test_norm_rope(debug_path, dt, D, rot, interleaved):  # noqa: F811
    g = torch.Generator().manual_seed(3)
    x = [torch.randn(2, h, 77, D, generator=g).to(dt).cuda() for h in (4, 2) * 4]
    w = [1 + 0.1 * torch.randn(D, generator=g).cuda() for _ in range(2)]
    kw = dict(rope=api.rope_table(80, rot, device="cuda"), q_weight=w[0], k_weight=w[1],
              interleaved=interleaved)
    both(debug_path, lambda: api.norm_rope(*x[:2], **kw))
    both(debug_path, lambda: api.norm_rope_dual(*x[:4], **kw))
    both(debug_path, lambda: api.norm_rope_bwd(*x[:4], **kw))
    both(debug_path, lambda: api.norm_rope_bwd_dual(*x, **kw))


@pytest.mark.parametrize("window,sinks", [(None, 0), (60, 3)])
@pytest.mark.parametrize("dt,H,Hkv,D,page,e4m3", [
    (torch.bfloat16, 8, 2, 128, 16, False), (torch.float16, 4, 4, 64, 24, False),
    (torch.bfloat16, 6, 2, 40, 5, False), (torch.bfloat16, 8, 2, 128, 16, True),
    (torch.float16, 4, 1, 64, 7, True), (torch.float32, 4, 2, 64, 16, False)])
def test_append_and_attend(debug_path, dt, H, Hkv, D, page, e4m3, window, sinks):  # noqa: F811
    new, past = [300, 1, 0, 70, 2], [900, 5000, 0, 3, 128]
    c = Cache([a + b for a, b in zip(new, past)], Hkv, D, page, dt, e4m3, 11)
    g = torch.Generator().manual_seed(5)
    x = [torch.randn(sum(new), h, D, generator=g).to(dt).cuda() for h in (H, Hkv, Hkv)]
    cu = torch.tensor([0] + new).cumsum(0).int().cuda()
    start, lens = (torch.tensor(n, dtype=torch.int32).cuda() for n in (past, c.lens))
    rope = api.rope_table(5100, D, device="cuda")

    def call():
        d = c.cuda()
        kw = dict(k_scale=d["k_scale"], v_scale=d["v_scale"])
        cache = (d["k_cache"], d["v_cache"], d["block_table"])
        q = api.cache_append(*x, *cache, rope, start, cu, **kw)
        o, lse = api.attention_chunk(q, *cache, lens, cu, window=window, sinks=sinks, return_lse=True, **kw)
        w = api.attention_decode(q[:5], *cache, lens, window=window, sinks=sinks, **kw)
        return q, o, lse, w, d["k_cache"].view(torch.uint8), d["v_cache"].view(torch.uint8)

    both(debug_path, call)
