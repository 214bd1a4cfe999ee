"""The native part of the binding on a GPU: errors, many layouts, threads with their own streams."""

import threading

import pytest
import torch

from forward_mode_flash_gb300 import api
from forward_mode_flash_gb300._abi import JvpAttnError

pytestmark = pytest.mark.gpu


def prompt(lens, H=4, Hkv=2, D=64, dt=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(sum(lens), h, D, generator=g).to(dt).cuda() for h in (H, Hkv, Hkv))
    return q, k, v, torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


def test_errors_of_the_library_and_of_the_arguments():
    q, k, v, cu = prompt([5, 9])
    with pytest.raises(JvpAttnError, match="scale is not finite"):
        api.attention_packed(q, k, v, cu, scale=float("inf"))
    with pytest.raises(TypeError):
        api.attention_packed(q, k, v, cu, scale="large")
    with pytest.raises(ValueError):
        api.attention_packed(q, k, v, cu.long())
    want = api.attention_packed(q, k, v, cu, scale=0.125)
    assert torch.equal(want, api.attention_packed(q, k, v, cu))
    assert torch.equal(want, api.attention_packed(q, k, v, cu, scale=torch.tensor(0.125)))


def test_a_workspace_is_checked_and_used():
    H, Hkv, D, page, B = 4, 2, 64, 16, 3
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.randn(120, Hkv, page, D, generator=g).half().cuda() for _ in range(2))
    q = torch.randn(B, H, D, generator=g).half().cuda()
    table = torch.arange(120, dtype=torch.int32).view(3, 40).cuda()
    lens = torch.tensor([600, 1, 640], dtype=torch.int32).cuda()
    n = api.decode_workspace_size(kc, table, H)
    assert n > 0
    want = api.attention_decode(q, kc, vc, table, lens)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(want, api.attention_decode(q, kc, vc, table, lens, workspace=ws))
    with pytest.raises(JvpAttnError, match="workspace"):
        api.attention_decode(q, kc, vc, table, lens, workspace=ws[:n - 1])
    with pytest.raises(ValueError):
        api.attention_decode(q, kc, vc, table, lens, workspace=ws.cpu())
    with pytest.raises(ValueError):
        api.attention_decode(q, kc, vc, table, lens, workspace=ws.repeat(2)[::2])


def test_more_layouts_than_are_remembered():
    q, k, v, cu = prompt([700])
    cu[1] = 1
    want = v[:1].repeat_interleave(2, 1)
    for T in list(range(1, 700)) + [1, 2, 3]:
        o = api.attention_packed(q[:T], k[:T], v[:T], cu)
        assert torch.equal(o[:1], want)


def test_threads_on_their_own_streams():
    work = [prompt([30 + 7 * i, 200, 1 + i], seed=i) for i in range(4)]
    want = [api.attention_packed(*w, is_causal=True) for w in work]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = api.attention_packed(*work[i], is_causal=True)
                if not torch.equal(got, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_split_calls_on_two_streams_at_once():
    """Each call has its own workspace, and so has each captured one."""
    H, Hkv, D, page = 8, 2, 128, 16
    g = torch.Generator().manual_seed(2)
    kc, vc = (torch.randn(800, Hkv, page, D, generator=g).bfloat16().cuda() for _ in range(2))
    qs = [torch.randn(2, H, D, generator=g).bfloat16().cuda() for _ in range(2)]
    tables = [torch.randperm(800, generator=g)[:600].view(2, 300).int().cuda() for _ in range(2)]
    lens = [torch.tensor(n, dtype=torch.int32).cuda() for n in ([4700, 800], [4800, 33])]
    assert api.decode_workspace_size(kc, tables[0], H) > 0
    calls = [lambda i=i: api.attention_decode(qs[i], kc, vc, tables[i], lens[i]) for i in range(2)]
    want = [c().clone() for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(100):
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
    for _ in range(50):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i])
    assert api.device_status() == 0
