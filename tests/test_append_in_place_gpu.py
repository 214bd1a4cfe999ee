"""Queries normalised and rotated in place on their rows' way into the cache."""

import pytest
import torch
from forward_mode_flash_gb300 import api, build

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# Rows of whole pieces, and layouts whose lanes read one another's columns: with columns
# that are not rotated, of fewer than a warp, of no whole number of warps, half a pair apart
# or next to one another.
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("cache", ["", "e4m3"])
@pytest.mark.parametrize("dt,D,rot", [("bf16", 128, 128), ("f32", 64, 32), ("f16", 80, 40), ("f32", 33, 6),
                                      ("bf16", 40, 20), ("f16", 24, 22), ("f32", 128, 2), ("bf16", 7, 4)])
def test_out_is_q(dt, D, rot, cache, norm, interleaved):
    T, H, Hkv, page = 3000, 6, 2, 16
    g = torch.Generator(device="cuda").manual_seed(D)
    # a projection's rows: queries, keys and values side by side
    qkv = torch.randn(T + 3, H + 2 * Hkv, D, generator=g, device="cuda").to(DT[dt])
    q, k, v = qkv.split((H, Hkv, Hkv), 1)
    pages = (T + page - 1) // page
    shape = (pages, Hkv, page, D)
    kind = torch.float8_e4m3fn if cache else DT[dt]
    caches = [torch.zeros(shape, device="cuda").to(kind) for _ in range(2)]
    scales = [torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") if cache else None
              for _ in range(2)]
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    w = [1 + 0.3 * torch.randn(D, generator=g, device="cuda") for _ in range(2)] if norm else [None] * 2
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = api.rope_table(T, rot, device="cuda")

    def append(q, k, v, **kw):
        return api.cache_append(q, k, v, *caches, table, rope, start, cu, *w, 1e-6, interleaved, *scales,
                                **kw)

    behind = qkv[T:].clone()
    want = append(q, k, v)[:T].clone()
    kept = [x.clone() for x in caches]
    for _ in range(3):
        rows = qkv.clone()
        a, b, c = rows.split((H, Hkv, Hkv), 1)
        got = append(a, b, c, out=a)
        assert got.data_ptr() == a.data_ptr() and torch.equal(got[:T], want)
        assert torch.equal(rows[T:], behind) and torch.equal(rows[:T, H:], qkv[:T, H:])
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(caches, kept))
