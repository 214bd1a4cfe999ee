"""The operators around the paged key-value cache, and the sizes they are measured at.

``attention_packed``: whole prompts of different lengths behind one another;
``attention_decode``: one new token per sequence against its cached keys;
``cache_write`` / ``cache_read``: rows into and out of the cache's pages, as
they are or in 8 bits (e4m3 with a power-of-two scale per row and head).

``run`` with ``own`` false computes each operator with elementary torch
operations in float32; with ``own`` true it calls the framework.  ``exact``
computes the same from the definition in float64.
"""

import math
import random

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
HEADS = ((8, 8), (16, 4), (16, 2), (8, 2), (12, 4), (16, 1), (6, 2))
E4M3_MAX = 448.0


def _case(name, op, sequences, shortest, longest, heads, kv_heads, dim, dtype, cache="", page=16,
          causal=True, mix=1):
    return {"name": name, "op": op, "sequences": sequences, "shortest": shortest,
            "longest": longest, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "cache": cache or dtype, "page": page, "causal": causal, "mix": mix}


def listed():
    return [
        # a few one-line prompts arriving together: latency counts
        _case("packed_short", "packed", 8, 1, 40, 8, 8, 64, "f16"),
        # an ordinary batch of prompts, grouped heads, no length a multiple of a tile
        _case("packed_ragged", "packed", 12, 37, 2048, 16, 4, 128, "bf16"),
        # two long documents
        _case("packed_long", "packed", 2, 9001, 16384, 16, 2, 128, "bf16"),
        # an encoder's batch, both directions
        _case("packed_both_ways", "packed", 16, 90, 1024, 8, 8, 64, "f16", causal=False),
        # full precision, for checking a model
        _case("packed_f32", "packed", 4, 61, 700, 8, 2, 64, "f32"),
        # one user, short context: latency counts
        _case("decode_one", "decode", 1, 130, 130, 16, 4, 128, "bf16"),
        # an ordinary serving batch of mixed lengths
        _case("decode_ragged", "decode", 48, 1, 4096, 16, 4, 128, "bf16"),
        # a large batch on an 8-bit cache
        _case("decode_e4m3", "decode", 64, 300, 16384, 16, 2, 128, "bf16", "e4m3", 64),
        # few users with very long contexts, one key head per query head
        _case("decode_long", "decode", 2, 70001, 131072, 8, 8, 64, "f16", page=32),
        # the step's new tokens into an 8-bit cache
        _case("write_step", "write", 48, 1, 4096, 16, 4, 128, "bf16", "e4m3"),
        # whole prompts into an 8-bit cache
        _case("write_prompts", "write", 12, 500, 8192, 16, 8, 128, "bf16", "e4m3", 64),
        # cached contexts back as dense keys and values
        _case("read_contexts", "read", 12, 500, 8192, 16, 8, 128, "bf16", "e4m3", 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("packed", "packed", "decode", "decode", "write", "read"))
    heads, kv_heads = rng.choice(HEADS)
    dim = rng.choice((64, 128, 128, 64, 96, 80, 40))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "packed":
        longest = _log(rng, 1, 8192 if dtype != "f32" else 1200)
        sequences = _log(rng, 1, max(1, min(64, 40000000 // longest ** 2)))
        cache = dtype
    else:
        longest = _log(rng, 1, 65536 if op == "decode" else 8192)
        sequences = _log(rng, 1, max(1, min(128, (1 << 17) // longest)))
        cache = rng.choice((dtype, "e4m3"))
    return {"op": op, "sequences": sequences, "shortest": rng.randint(1, longest),
            "longest": longest, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "cache": cache, "page": rng.choice((8, 16, 32, 64, 128, 24, 1)) if longest < 20000
            else 64, "causal": rng.random() < 0.7, "mix": rng.randint(1, 1 << 20)}


def _lengths(case):
    """Each sequence's length: the longest first, then spread between the bounds."""
    rng = random.Random(case["mix"])
    lo, hi = case["shortest"], case["longest"]
    return [hi] + [rng.randint(lo, hi) for _ in range(case["sequences"] - 1)]


def _rows(case):
    """How many rows of each sequence a call handles (a write of single tokens: one)."""
    n = _lengths(case)
    return [1] * len(n) if case["op"] == "write" and case["shortest"] == 1 else n


def work(case):
    n, rows = _lengths(case), sum(_rows(case))
    H, Hk, D, e = case["heads"], case["kv_heads"], case["dim"], SIZE[case["dtype"]]
    row = 2 * Hk * D * SIZE[case["cache"]] + (2 * Hk if case["cache"] == "e4m3" else 0)
    if case["op"] == "packed":
        pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in n)
        return {"bytes": rows * ((2 * H + 2 * Hk) * D * e + 4 * H), "flops": 4 * D * H * pairs}
    if case["op"] == "decode":
        return {"bytes": rows * row + len(n) * H * (2 * D * e + 4), "flops": 4 * D * H * rows}
    return {"bytes": rows * (row + 2 * Hk * D * e), "flops": 0}


def _quantise(x):
    """Codes and scale bytes: the smallest power of two 2^e with max|x| <= 448 * 2^e."""
    x = x.float()
    top = x.abs().amax(-1)
    fraction, power = torch.frexp(top)  # top = fraction * 2^power, fraction in [0.5, 1)
    e = torch.where(fraction * 2 <= E4M3_MAX / 256, power - 9, power - 8)
    e = torch.where(top > 0, e, -127).clamp(-127, 127)
    codes = torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, scale):
    """What a cache holds: its entries, times their scale where there is one."""
    x = codes.float()
    return x if scale is None else torch.ldexp(x, scale.int().unsqueeze(-1) - 127)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    n, rows = _lengths(case), _rows(case)
    B, T = len(n), sum(rows)
    H, Hk, D, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    dt = DTYPE[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(rows).cumsum(0)
    state = {"case": case, "longest": max(n), "cu": cu.to(dev),
             "row_of": torch.cat([torch.arange(r) for r in rows]).to(dev),
             "sequence_of": torch.repeat_interleave(torch.arange(B), torch.tensor(rows)).to(dev)}
    if case["op"] == "packed":
        state.update(q=normal(T, H, D), k=normal(T, Hk, D), v=normal(T, Hk, D))
        return state
    # pages in no order; entries behind a sequence's last page are -1
    need = [-(-x // page) for x in n]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    shape = (pages, Hk, page, D)
    e4m3 = case["cache"] == "e4m3"
    state.update(table=table, lens=torch.tensor(n, dtype=torch.int32, device=dev), ks=None, vs=None)
    # a row is where its call's first row lands plus its place in the call
    state["start"] = (state["lens"] - torch.tensor(rows, dtype=torch.int32, device=dev))
    if case["op"] == "write":
        kind = torch.float8_e4m3fn if e4m3 else DTYPE[case["cache"]]
        state.update(k=normal(T, Hk, D), v=normal(T, Hk, D),
                     kc=torch.zeros(shape, device=dev).to(kind),
                     vc=torch.zeros(shape, device=dev).to(kind))
        if e4m3:
            state.update(ks=torch.zeros(shape[:3], dtype=torch.uint8, device=dev),
                         vs=torch.zeros(shape[:3], dtype=torch.uint8, device=dev))
        return state
    kc, vc = normal(*shape), normal(*shape)
    if e4m3:
        (kc, state["ks"]), (vc, state["vs"]) = _quantise(kc), _quantise(vc)
    state.update(kc=kc, vc=vc)
    if case["op"] == "decode":
        state["q"] = normal(B, H, D)
    return state


def _attend(q, k, v, keep, scale):
    """Softmax attention of [.., M, D] on [.., N, D] over the kept pairs, and its log-sum-exp."""
    s = torch.matmul(q * scale, k.transpose(-1, -2))
    s.masked_fill_(~keep, -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    return torch.matmul(s, v) / total, (m + total.log()).squeeze(-1)


def _plain_packed(st):
    case, N, cu = st["case"], st["longest"], st["cu"].long()
    T, H, D = st["q"].shape
    Hk, B = st["k"].shape[1], len(cu) - 1
    place = torch.arange(N, device=cu.device)
    lens = cu[1:] - cu[:-1]
    take = (cu[:-1, None] + place).clamp_(max=T - 1)  # padded to the longest
    q = st["q"].float()[take].view(B, N, Hk, H // Hk, D).permute(0, 2, 3, 1, 4)
    k, v = (st[x].float()[take].permute(0, 2, 1, 3).unsqueeze(2) for x in ("k", "v"))
    keep = (place < lens[:, None]).view(B, 1, 1, 1, N)
    if case["causal"]:
        keep = keep & (place <= place[:, None])
    o, lse = _attend(q, k, v, keep, 1.0 / math.sqrt(D))
    b, i = st["sequence_of"], st["row_of"]
    return {"o": o[b, :, :, i].reshape(T, H, D).to(st["q"].dtype),
            "lse": lse[b, :, :, i].reshape(T, H).t().contiguous()}


def _plain_decode(st):
    B, H, D = st["q"].shape
    _, Hk, page, _ = st["kc"].shape
    table = st["table"].clamp(min=0).long()
    N = table.shape[1] * page

    def dense(cache, scale):
        x = _values(cache[table], None if scale is None else scale[table])
        return x.transpose(1, 2).reshape(B, Hk, N, D)

    keep = (torch.arange(N, device=table.device) < st["lens"][:, None]).view(B, 1, 1, N)
    o, lse = _attend(st["q"].float().view(B, Hk, H // Hk, D), dense(st["kc"], st["ks"]),
                     dense(st["vc"], st["vs"]), keep, 1.0 / math.sqrt(D))
    return {"o": o.reshape(B, H, D).to(st["q"].dtype), "lse": lse.reshape(B, H)}


def _slots(st):
    """Page and place in it of every row of a call."""
    page = st["kc"].shape[2]
    position = st["start"].long()[st["sequence_of"]] + st["row_of"]
    return st["table"][st["sequence_of"], position // page].long(), position % page


def _plain_write(st):
    at, place = _slots(st)
    for x, cache, scale in (("k", "kc", "ks"), ("v", "vc", "vs")):
        if st[scale] is None:
            st[cache][at, :, place] = st[x]
        else:
            codes, s = _quantise(st[x])
            st[cache].view(torch.uint8)[at, :, place] = codes.view(torch.uint8)
            st[scale][at, :, place] = s
    return _cache(st)


def _cache(st):
    return {x: st[x] for x in ("kc", "vc", "ks", "vs") if st[x] is not None}


def _plain_read(st):
    at, place = _slots(st)
    dt = DTYPE[st["case"]["dtype"]]

    def rows(cache, scale):
        return _values(cache[at, :, place], None if scale is None else scale[at, :, place]).to(dt)

    return {"k": rows(st["kc"], st["ks"]), "v": rows(st["vc"], st["vs"])}


def _own(st):
    from forward_mode_flash_gb300 import api

    case = st["case"]
    if case["op"] == "packed":
        o, lse = api.attention_packed(st["q"], st["k"], st["v"], st["cu"],
                                      is_causal=case["causal"], return_lse=True)
        return {"o": o, "lse": lse}
    if case["op"] == "decode":
        o, lse = api.attention_decode(st["q"], st["kc"], st["vc"], st["table"], st["lens"],
                                      k_scale=st["ks"], v_scale=st["vs"], return_lse=True)
        return {"o": o, "lse": lse}
    if case["op"] == "write":
        api.cache_write(st["k"], st["v"], st["kc"], st["vc"], st["table"], st["start"], st["cu"],
                        k_scale=st["ks"], v_scale=st["vs"])
        return _cache(st)
    k, v = api.cache_read(st["kc"], st["vc"], st["table"], st["start"], st["cu"],
                          num_rows=len(st["row_of"]), k_scale=st["ks"], v_scale=st["vs"],
                          dtype=DTYPE[case["dtype"]])
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    return {"packed": _plain_packed, "decode": _plain_decode, "write": _plain_write,
            "read": _plain_read}[state["case"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits
def _softmax_64(q, k, v, causal):
    """Attention of one head, query rows in blocks; q, k, v float64."""
    o, lse = [], []
    for r in range(0, len(q), 4096):
        logits = q[r:r + 4096] @ k.T / math.sqrt(q.shape[1])
        if causal:
            i = torch.arange(r, r + len(logits), device=q.device)
            logits[torch.arange(len(k), device=q.device) > i[:, None]] = -math.inf
        z = torch.logsumexp(logits, 1)
        o.append((logits - z[:, None]).exp() @ v)
        lse.append(z)
    return torch.cat(o), torch.cat(lse)


def _gather_64(st, cache, scale, b, positions, head):
    """One head's cached rows of a sequence, as values."""
    page = cache.shape[2]
    at = st["table"][b].long()[positions // page]
    x = cache[at, head, positions % page].double()
    if scale is not None:
        x = x * torch.exp2(scale[at, head, positions % page].double() - 127)[:, None]
    return x


def _round_e4m3(y):
    """The nearest e4m3 value (ties to even) of float64 numbers of magnitude up to 464."""
    power = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(power - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    dev = st["cu"].device
    n = _lengths(case)
    if case["op"] == "packed":
        o = torch.zeros(sum(n), H, D, dtype=torch.float64, device=dev)
        lse = torch.zeros(H, sum(n), dtype=torch.float64, device=dev)
        first = 0
        for length in n:
            r = slice(first, first + length)
            for h in range(H):
                hk = h // (H // Hk)
                o[r, h], lse[h, r] = _softmax_64(st["q"][r, h].double(), st["k"][r, hk].double(),
                                                 st["v"][r, hk].double(), case["causal"])
            first += length
        return {"o": o, "lse": lse}
    if case["op"] == "decode":
        o = torch.zeros(len(n), H, D, dtype=torch.float64, device=dev)
        lse = torch.zeros(len(n), H, dtype=torch.float64, device=dev)
        for b, length in enumerate(n):
            every = torch.arange(length, device=dev)
            for hk in range(Hk):
                r = slice(hk * (H // Hk), (hk + 1) * (H // Hk))
                o[b, r], lse[b, r] = _softmax_64(st["q"][b, r].double(),
                                                 _gather_64(st, st["kc"], st["ks"], b, every, hk),
                                                 _gather_64(st, st["vc"], st["vs"], b, every, hk),
                                                 False)
        return {"o": o, "lse": lse}
    first = 0
    if case["op"] == "read":
        k, v = (torch.zeros(sum(n), Hk, D, dtype=torch.float64, device=dev) for _ in range(2))
        for b, length in enumerate(n):
            every = torch.arange(length, device=dev)
            for hk in range(Hk):
                k[first:first + length, hk] = _gather_64(st, st["kc"], st["ks"], b, every, hk)
                v[first:first + length, hk] = _gather_64(st, st["vc"], st["vs"], b, every, hk)
            first += length
        return {"k": k, "v": v}
    out = {x: st[x].double() if x in ("kc", "vc") else st[x].clone() for x in _cache(st)}
    for b, rows in enumerate(_rows(case)):
        position = n[b] - rows + torch.arange(rows, device=dev)
        at, place = st["table"][b].long()[position // case["page"]], position % case["page"]
        for x, cache, scale in (("k", "kc", "ks"), ("v", "vc", "vs")):
            y = st[x][first:first + rows].double()
            if st[scale] is not None:
                e = torch.ceil(torch.log2(y.abs().amax(-1) / E4M3_MAX)).clamp(-127, 127)
                y = _round_e4m3(y / torch.exp2(e)[..., None])
                out[scale][at, :, place] = (e + 127).to(torch.uint8)
            out[cache][at, :, place] = y
        first += rows
    return out
