"""Rows appended with norms and rotation, attention of chunks over them and single tokens with a
window: run one after the other, as a server does, against the definition in float64."""

import numpy as np
import pytest
import torch

from forward_mode_flash_gb300 import _abi, api, build
from serving_ref import attend, bounds, f64

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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


class Server:
    """Sequences whose rows go into a paged cache step by step; `said` holds all rows of each."""

    def __init__(self, B, H, Hkv, D, dt, page, e4m3, most, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        cols = -(-most // page)
        kt = torch.float8_e4m3fn if e4m3 else DT[dt]
        self.kc, self.vc = (torch.zeros(B * cols, Hkv, page, D, device="cuda").to(kt) for _ in range(2))
        self.sc = [torch.full((B * cols, Hkv, page), 127, dtype=torch.uint8, device="cuda") if e4m3
                   else None for _ in range(2)]
        self.table = torch.randperm(B * cols, generator=self.g).view(B, cols).int().cuda()
        self.rope = api.rope_table(most, D, device="cuda")
        self.w = [1 + 0.2 * torch.randn(D, generator=self.g).cuda() for _ in range(2)]
        self.H, self.Hkv, self.D, self.dt, self.lens = H, Hkv, D, DT[dt], [0] * B
        self.said = [[torch.zeros(0, h, D, dtype=self.dt) for _ in range(B)] for h in (H, Hkv, Hkv)]

    def rows(self, new):
        x = [torch.randn(sum(new), h, self.D, generator=self.g).to(self.dt)
             for h in (self.H, self.Hkv, self.Hkv)]
        at = 0
        for b, n in enumerate(new):
            for s, y in zip(self.said, x):
                s[b] = torch.cat((s[b], y[at:at + n]))
            at += n
        return [y.cuda() for y in x]

    def append(self, x, new, past, single=False):
        cu = None if single else i32(np.concatenate([[0], np.cumsum(new)]))
        return api.cache_append(*x, self.kc, self.vc, self.table, self.rope, i32(past), cu, *self.w,
                                k_scale=self.sc[0], v_scale=self.sc[1])

    def step(self, new, window=None, sinks=0, single=False):
        past, self.lens = self.lens, [a + b for a, b in zip(self.lens, new)]
        q = self.append(self.rows(new), new, past, single)
        kw = dict(window=window, sinks=sinks, k_scale=self.sc[0], v_scale=self.sc[1], return_lse=True)
        if single:
            o, lse = api.attention_decode(q, self.kc, self.vc, self.table, i32(self.lens), **kw)
            lse = lse.t()
        else:
            cu = i32(np.concatenate([[0], np.cumsum(new)]))
            o, lse = api.attention_chunk(q, self.kc, self.vc, self.table, i32(self.lens), cu, **kw)
        self.check(new, q, o, lse, window, sinks, api.last_path() == 1)

    def check(self, new, q, o, lse, window, sinks, tc):
        G, D, at = self.H // self.Hkv, self.D, 0
        u = torch.finfo(self.dt).eps / 2
        for b, n in enumerate(new):
            if n == 0:
                continue
            # queries and the cache's rows are the dense operator's
            one = [s[b].transpose(0, 1)[None].cuda() for s in self.said]
            rq, rk = api.norm_rope(one[0], one[1], self.rope, None, *self.w)
            assert torch.equal(q[at:at + n], rq[0].transpose(0, 1)[-n:])
            total = self.lens[b]
            k, v = api.cache_read(self.kc, self.vc, self.table[b:b + 1], None, i32([0, total]),
                                  num_rows=total, dtype=self.dt, k_scale=self.sc[0], v_scale=self.sc[1])
            if self.sc[0] is None:
                assert torch.equal(k, rk[0].transpose(0, 1)) and torch.equal(v, one[2][0].transpose(0, 1))
            x, j = total - n + np.arange(n), np.arange(total)
            keep = j <= x[:, None]
            if window is not None:
                keep &= (j > x[:, None] - window) | (j < sinks)
            for h in range(self.H):
                ref = attend(f64(q[at:at + n, h]), f64(k[:, h // G]), f64(v[:, h // G]), keep, D ** -0.5)
                b_o, b_lse = bounds(*ref, total, D, u, u if tc else 0.0, tc)
                assert (np.abs(f64(o[at:at + n, h]) - ref[0]) <= b_o).all(), (b, h)
                assert (np.abs(f64(lse[h, at:at + n]) - ref[1]) <= b_lse).all(), (b, h)
            at += n


@pytest.mark.parametrize("window,sinks", [(None, 0), (48, 4)])
@pytest.mark.parametrize("dt,H,Hkv,D,page,e4m3", [
    ("bf16", 8, 2, 128, 16, False), ("f16", 4, 4, 64, 24, False), ("bf16", 6, 2, 64, 5, False),
    ("bf16", 8, 2, 128, 16, True), ("f32", 4, 2, 64, 16, False), ("bf16", 4, 1, 64, 3, True)])
def test_prompts_chunks_and_single_tokens(dt, H, Hkv, D, page, e4m3, window, sinks):
    s = Server(4, H, Hkv, D, dt, page, e4m3, 400, seed=D + page)
    s.step([150, 1, 30, 0], window, sinks)   # prompts
    s.step([40, 129, 0, 7], window, sinks)   # the rest of some, and a new one
    s.step([4, 4, 4, 4], window, sinks)      # drafted tokens
    for _ in range(3):
        s.step([1, 1, 1, 1], window, sinks, single=True)
    s.step([0, 200, 1, 3], window, sinks)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_captured_step_is_replayed_for_every_token(e4m3):
    """Append, chunk and single tokens captured together; each replay is the eager step."""
    B, H, Hkv, D, page, most = 3, 8, 2, 128, 16, 600
    s = [Server(B, H, Hkv, D, "bf16", page, e4m3, most, seed=1) for _ in range(2)]
    new = [200, 1, 350]
    for x in s:
        x.step(new, 100, 3)
    lens, start = i32(new), i32(new)
    cu = i32([0, 2, 4, 6])
    x = [torch.zeros(2 * B, h, D, device="cuda", dtype=torch.bfloat16) for h in (H, Hkv, Hkv)]

    def step(t):
        kw = dict(window=100, sinks=3, k_scale=t.sc[0], v_scale=t.sc[1])
        q = api.cache_append(*x, t.kc, t.vc, t.table, t.rope, start, cu, *t.w, k_scale=t.sc[0],
                             v_scale=t.sc[1])
        o = api.attention_chunk(q, t.kc, t.vc, t.table, lens, cu, **kw)
        return o, api.attention_decode(q[1::2], t.kc, t.vc, t.table, lens, **kw)

    lens += 2
    keep = [c.clone() for c in (s[0].kc, s[0].vc)]
    step(s[0])
    for c, k in zip((s[0].kc, s[0].vc), keep):
        c.copy_(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s[0])
    g = torch.Generator().manual_seed(5)
    for i in range(4):
        for t in x:
            t.copy_(torch.randn(t.shape, generator=g))
        graph.replay()
        for a, b in zip(got, step(s[1])):
            assert torch.equal(a, b), i
        # The last of each chunk is a single token too: each kernel rounds its weights and its
        # output once, by 2^-8 of values below 6 (e4m3 rows included).
        assert (got[0][1::2].float() - got[1].float()).abs().max() <= 4 * 2 ** -8 * 6
        lens += 2
        start += 2


def test_chunks_on_two_streams_and_in_two_graphs():
    """Each call has its own workspace, and so has each captured one."""
    g = torch.Generator().manual_seed(2)
    H, Hkv, D, page = 8, 2, 128, 16
    kc, vc = (torch.randn(800, Hkv, page, D, generator=g).bfloat16().cuda() for _ in range(2))
    qs = [torch.randn(n, H, D, generator=g).bfloat16().cuda() for n in (9, 150)]
    tables = [torch.randperm(800, generator=g)[:600].view(2, 300).int().cuda() for _ in range(2)]
    lens = [i32([4700, 800]), i32([4800, 133])]
    cus = [i32([0, 5, 9]), i32([0, 100, 150])]
    calls = [lambda i=i: api.attention_chunk(qs[i], kc, vc, tables[i], lens[i], cus[i]) for i in range(2)]
    assert all(api.chunk_workspace_size(qs[i], kc, tables[i]) > 0 for i in range(2))
    want = [c().clone() for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(60):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(calls[i]())
        graphs.append(graph)
    for _ in range(40):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i])


@pytest.mark.parametrize("dt,page,e4m3", [("bf16", 16, False), ("bf16", 12, False), ("bf16", 16, True),
                                          ("bf16", 12, True), ("f32", 16, False)])
def test_places_beyond_31_bits(dt, page, e4m3):
    """The last pages of a cache of more than 2^31 elements give what the first of a small one do."""
    H, Hkv, D, B = 4, 2, 64, 2
    per = 2 ** 31 // (Hkv * page * D) + 40
    kt = torch.float8_e4m3fn if e4m3 else DT[dt]
    new, past = [70, 3], [200, 430]
    cols = -(-440 // page)
    g = torch.Generator().manual_seed(7)
    x = [torch.randn(sum(new), h, D, generator=g).to(DT[dt]).cuda() for h in (H, Hkv, Hkv)]
    old = [torch.randn(B * cols, Hkv, page, D, generator=g).cuda().to(kt) for _ in range(2)]
    rope = api.rope_table(512, D, device="cuda")
    small = torch.randperm(B * cols, generator=g).view(B, cols).int().cuda()
    cu, start, lens = i32([0, 70, 73]), i32(past), i32([a + b for a, b in zip(new, past)])
    out = []
    for first in (0, per):  # the first page
        kc, vc = (torch.empty(first + B * cols, Hkv, page, D, dtype=kt, device="cuda") for _ in range(2))
        kc[first:], vc[first:] = old
        sc = [torch.full(kc.shape[:3], 126, dtype=torch.uint8, device="cuda") if e4m3 else None
              for _ in range(2)]
        kw = dict(k_scale=sc[0], v_scale=sc[1])
        table = small + first
        q = api.cache_append(*x, kc, vc, table, rope, start, cu, **kw)
        o, lse = api.attention_chunk(q, kc, vc, table, lens, cu, return_lse=True, **kw)
        w = api.attention_decode(q[[69, 72]], kc, vc, table, lens, window=90, sinks=2, **kw)
        out.append([q, o, lse, w, kc[first:].view(torch.uint8).clone(), vc[first:].view(torch.uint8).clone()])
        del kc, vc, sc
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_rows_beyond_31_bits():
    """Queries and outputs of more than 2^31 elements."""
    H, D, T = 128, 128, 2 ** 17 + 300
    g = torch.Generator().manual_seed(3)
    q = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    q[-250:] = torch.randn(250, H, D, generator=g).cuda()
    kc, vc = (torch.randn(40, 8, 16, D, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.arange(40, dtype=torch.int32).view(1, 40).cuda()
    want = api.attention_chunk(q[-250:].clone(), kc, vc, table, i32([640]), i32([0, 250]))
    o = api.attention_chunk(q, kc, vc, table, i32([640]), i32([T - 250, T]))
    assert torch.equal(o[-250:], want)
