"""Offsets of cache_write and cache_read that are out of range: reported, and
their sequences skipped."""

import numpy as np
import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(autouse=True)
def _status_clear():
    api.device_status()
    yield
    assert api.device_status() == _abi.JVP_OK


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


# offsets, and the sequences whose rows must be in their places
BAD = [
    ([0, 50, 40, 40], [0]),          # a length below 0
    ([0, 50, 20, 60], [0]),          # overlapping sequences (of the third nothing is promised)
    ([-5, 50, 110, 150], [1, 2]),    # a start in front of the rows
    ([0, 50, 110, 151], [0, 1]),     # an end behind them
    ([0, 50, 110, 2 ** 31 - 1], [0, 1]),
    ([-2 ** 31, -1, 110, 150], [2]),
    ([0, 150, 0, 150], [0]),
]


@pytest.mark.parametrize("e4m3,D", [(False, 64), (True, 64), (False, 33), (True, 33)])
@pytest.mark.parametrize("cu,good", BAD)
def test_bad_offsets_are_skipped_and_reported(cu, good, e4m3, D):
    T, Hkv, page, most = 150, 2, 16, 12
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(T, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc, vc = (torch.full((3 * most + 1, Hkv, page, D), 3.0, device="cuda").to(dt) for _ in range(2))
    sc = [torch.full(kc.shape[:3], 127, dtype=torch.uint8, device="cuda") if e4m3 else None
          for _ in range(2)]
    table = torch.randperm(3 * most, generator=g).int().view(3, most).cuda()
    kw = dict(k_scale=sc[0], v_scale=sc[1])
    api.cache_write(k, v, kc, vc, table, None, i32(cu), **kw)
    assert api.device_status() == _abi.JVP_ERR_INDEX

    def held(b, n):
        return api.cache_read(kc, vc, table[b:b + 1], None, i32([0, n]), num_rows=n, **kw)

    # what the same rows are as a sequence of their own, in another cache
    other = [torch.zeros_like(x) for x in (kc, vc)]
    osc = [torch.zeros_like(s) if e4m3 else None for s in sc]
    okw = dict(k_scale=osc[0], v_scale=osc[1])
    touched = torch.zeros(3, most * page, dtype=torch.bool)
    for b in range(3):
        r0, r1 = cu[b], cu[b + 1]
        if not 0 <= r0 <= r1 <= T:
            continue
        n = r1 - r0
        touched[b, :n] = True
        if b in good and n:
            api.cache_write(k[r0:r1], v[r0:r1], *other, table[b:b + 1], None, i32([0, n]), **okw)
            want = api.cache_read(*other, table[b:b + 1], None, i32([0, n]), num_rows=n, **okw)
            for x, y in zip(held(b, n), want):
                assert torch.equal(x, y)
    # nothing else has been written
    for b in range(3):
        for x in held(b, most * page):
            assert x[~touched[b].cuda()].eq(3.0).all()
    assert kc[3 * most].float().eq(3.0).all() and vc[3 * most].float().eq(3.0).all()
    assert api.device_status() == _abi.JVP_OK

    # reading by the same offsets
    every = i32(np.arange(4) * most * page)
    all_k, _ = api.cache_read(kc, vc, table, None, every, num_rows=3 * most * page, **kw)
    out = tuple(torch.full((T, Hkv, D), 9.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    api.cache_read(kc, vc, table, None, i32(cu), out=out, **kw)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    covered = torch.zeros(T, dtype=torch.bool)
    for b in range(3):
        r0, r1 = cu[b], cu[b + 1]
        if 0 <= r0 <= r1 <= T:
            covered[r0:r1] = True
            if b in good:
                assert torch.equal(out[0][r0:r1], all_k[b * most * page:][:r1 - r0])
    for x in out:
        assert x[~covered.cuda()].eq(9.0).all()


def test_too_few_rows_for_the_offsets_are_reported():
    kc = torch.ones(4, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    table = i32([[0, 1], [2, 3]])
    out = tuple(torch.full((30, 1, 64), 9.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    api.cache_read(kc, kc, table, None, i32([0, 20, 40]), out=out)
    assert api.device_status() == _abi.JVP_ERR_INDEX
    assert out[0][:20].eq(1.0).all() and out[0][20:].eq(9.0).all()


@pytest.mark.parametrize("where", [1, 31, 32, 33, 500, 999])
@pytest.mark.parametrize("rows", [1, 3, 400])
def test_every_offset_is_looked_at(rows, where):
    """More sequences than the rows' threads (and fewer): one offset is wrong."""
    B = 1000
    kc = torch.zeros(2, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    x = torch.ones(rows, 1, 64, device="cuda", dtype=torch.bfloat16)
    table = torch.zeros(B, 25, dtype=torch.int32, device="cuda")
    cu = np.zeros(B + 1)
    cu[B] = min(rows, 16)
    api.cache_write(x, x, kc, kc.clone(), table, None, i32(cu))
    assert api.device_status() == _abi.JVP_OK
    cu[where] = -1
    api.cache_write(x, x, kc, kc.clone(), table, None, i32(cu))
    assert api.device_status() == _abi.JVP_ERR_INDEX


def test_padded_batches_are_in_order():
    """Rows in front of the first sequence and behind the last are nobody's."""
    kc = torch.zeros(2, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    x = torch.ones(12, 1, 64, device="cuda", dtype=torch.bfloat16)
    api.cache_write(x, x, kc, kc.clone(), i32([[0], [1]]), None, i32([3, 3, 8]))
    assert api.device_status() == _abi.JVP_OK
    assert kc[1, 0, :5].eq(1).all() and kc[1, 0, 5:].eq(0).all() and kc[0].eq(0).all()
