"""The operators between projections and attention, and attention over cached
contexts of more than one new token or within a window; the sizes they are measured at.

``attention_chunk``: some new tokens of each sequence against its paged cache,
with a sliding window and first tokens that stay visible, or without;
``attention_decode`` with such a window: one new token per sequence;
``cache_append``: queries and keys normalised per head and rotated by their
positions, keys and values into the cache's pages;
``norm_rope``: the same norms and rotation on dense tensors for training, with
their tangents and gradients.

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
EPS = 1e-6


def _chunk(name, sequences, new, past, heads, kv_heads, dim, dtype, cache="", page=16, window=0,
           sinks=0, mix=1):
    return {"name": name, "op": "chunk", "sequences": sequences, "new_lo": new[0], "new_hi": new[1],
            "past_lo": past[0], "past_hi": past[1], "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "cache": cache or dtype, "page": page, "window": window,
            "sinks": sinks, "mix": mix}


def _decode(name, sequences, past, heads, kv_heads, dim, dtype, cache="", page=16, window=0,
            sinks=0, mix=1):
    case = _chunk(name, sequences, (1, 1), past, heads, kv_heads, dim, dtype, cache, page, window,
                  sinks, mix)
    return {**case, "op": "decode"}


def _append(name, sequences, new, past, heads, kv_heads, dim, dtype, rotary, norm, interleaved=False,
            page=16, mix=1):
    case = _chunk(name, sequences, new, past, heads, kv_heads, dim, dtype, dtype, page, mix=mix)
    return {**case, "op": "append", "rotary": rotary, "norm": norm, "interleaved": interleaved}


def _norm(name, tangents, batch, tokens, heads, kv_heads, dim, dtype, rotary, interleaved=False):
    return {"name": name, "op": "norm", "tangents": tangents, "sequences": batch, "tokens": tokens,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "rotary": rotary,
            "interleaved": interleaved}


def listed():
    return [
        # a few drafted tokens per user to be verified: latency and the cache's bytes count
        _chunk("chunk_draft", 32, (1, 8), (100, 8192), 16, 4, 128, "bf16"),
        # the next pieces of two long documents
        _chunk("chunk_prefill", 2, (2000, 4096), (9001, 16384), 16, 2, 128, "bf16", page=64),
        # a continuous batch: some users at single tokens, some in the middle of a prompt
        _chunk("chunk_mixed", 24, (1, 512), (1, 4096), 16, 4, 128, "bf16"),
        # long prompts of a model with a window of 1024 tokens and four that stay visible
        _chunk("chunk_window", 3, (1500, 6000), (0, 5000), 8, 8, 64, "f16", page=32, window=1024,
               sinks=4),
        # pieces of prompts over an 8-bit cache
        _chunk("chunk_e4m3", 8, (64, 512), (500, 8192), 16, 4, 128, "bf16", "e4m3", 64),
        # full precision, for checking a model; some keys per query masked by a small window
        _chunk("chunk_f32", 4, (0, 300), (17, 700), 8, 2, 64, "f32", window=200, sinks=2),
        # one user, a short window: latency counts
        _decode("decode_window_one", 1, (5000, 5000), 16, 4, 128, "bf16", window=512, sinks=4),
        # a serving batch far beyond its window
        _decode("decode_window", 64, (100, 32768), 16, 4, 128, "bf16", page=64, window=4096,
                sinks=16),
        # the step's new tokens, rotated into the cache
        _append("append_step", 48, (1, 1), (0, 4096), 16, 4, 128, "bf16", 128, True),
        # whole prompts, half of each head rotated, no norms
        _append("append_prompts", 12, (500, 8192), (0, 0), 16, 8, 128, "bf16", 64, False, page=64),
        # a training step's queries and keys, forwards and backwards
        _norm("norm_train", False, 4, 4096, 16, 4, 128, "bf16", 128),
        # the same with tangents, in full precision
        _norm("norm_tangents", True, 2, 1531, 8, 8, 64, "f32", 64, interleaved=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "chunk", "decode", "append", "norm"))
    heads, kv_heads = rng.choice(HEADS)
    dim = rng.choice((64, 128, 128, 64, 96, 80, 40))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    page = rng.choice((8, 16, 32, 64, 128, 24, 1))
    window = rng.choice((0, 0, _log(rng, 1, 4096)))
    sinks = rng.choice((0, 1, 4, 130)) if window else 0
    cache = rng.choice((dtype, dtype, "e4m3"))
    rotary = rng.choice((dim, dim, dim // 2))
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "mix": rng.randint(1, 1 << 20)}
    if op == "norm":
        tokens = _log(rng, 1, 8192)
        return {**case, "tangents": rng.random() < 0.5, "tokens": tokens,
                "sequences": _log(rng, 1, max(1, min(64, 16384 // tokens))), "rotary": rotary,
                "interleaved": rng.random() < 0.3}
    if op == "decode":
        past = _log(rng, 1, 65536)
        sequences = _log(rng, 1, max(1, min(128, (1 << 18) // past)))
        new = 1
        window, sinks = (window, sinks) if window else (_log(rng, 1, 4096), 4)
    elif op == "append":
        past, new = _log(rng, 1, 8192), _log(rng, 1, 8192)
        sequences = _log(rng, 1, max(1, min(128, (1 << 16) // new)))
        cache = dtype
    else:
        new = _log(rng, 1, 4096 if dtype != "f32" else 400)
        past = _log(rng, 1, 16384 if dtype != "f32" else 1500)
        sequences = _log(rng, 1, max(1, min(64, 60000000 // (new * (past + new)))))
    case.update(sequences=sequences, new_lo=1 if op == "decode" else rng.randint(0, new), new_hi=new,
                past_lo=rng.randint(0, past), past_hi=past, cache=cache,
                page=page if past + new < 20000 else 64, window=window, sinks=sinks)
    if op == "append":
        case.update(rotary=rotary, norm=rng.random() < 0.6, interleaved=rng.random() < 0.3)
    return case


def _lengths(case):
    """Each sequence's new tokens and those before: the longest first, then spread, with
    some of the sequences at the fewest new tokens."""
    rng = random.Random(case["mix"])
    lo, hi = case["new_lo"], case["new_hi"]
    new = [hi] + [lo if rng.random() < 0.4 else rng.randint(lo, hi)
                  for _ in range(case["sequences"] - 1)]
    past = [case["past_hi"]] + [rng.randint(case["past_lo"], case["past_hi"])
                                for _ in range(case["sequences"] - 1)]
    return new, past


def work(case):
    H, Hk, D, e = case["heads"], case["kv_heads"], case["dim"], SIZE[case["dtype"]]
    if case["op"] == "norm":
        rows = case["sequences"] * case["tokens"] * (H + Hk)
        # x in and y out; x, gy in and gx out; as many again for the tangents
        return {"bytes": rows * D * e * 5 * (2 if case["tangents"] else 1),
                "flops": rows * D * (60 if case["tangents"] else 25)}
    new, past = _lengths(case)
    if case["op"] == "append":
        return {"bytes": sum(new) * D * e * (2 * H + 4 * Hk), "flops": sum(new) * D * 8 * (H + Hk)}
    W, S = case["window"], case["sinks"]
    cached = pairs = 0
    for n, p in zip(new, past):
        if not n:
            continue
        first, last = p, p + n - 1  # positions of its first and last new token
        if not W:
            cached, pairs = cached + last + 1, pairs + n * (first + last + 2) // 2
            continue
        # rows that some token sees: those after first - W, and the sinks before them
        lo = max(0, first - W + 1)
        cached += last + 1 - lo + min(S, lo)
        for q in range(first, last + 1):
            lo = max(0, q - W + 1)
            pairs += q + 1 - lo + min(S, lo)
    row = 2 * Hk * D * SIZE[case["cache"]] + (2 * Hk if case["cache"] == "e4m3" else 0)
    return {"bytes": cached * row + sum(new) * H * (2 * D * e + 4), "flops": 4 * D * H * pairs}


def _quantise(x):
    """Codes and scale bytes: the smallest power of two 2^e with max|x| <= 448 * 2^e."""
    x = x.float()
    top = x.abs().amax(-1)
    fraction, power = torch.frexp(top)  # top = fraction * 2^power, fraction in [0.5, 1)
    e = torch.where(fraction * 2 <= 448.0 / 256, power - 9, power - 8)
    e = torch.where(top > 0, e, -127).clamp(-127, 127)
    codes = torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _angles(positions, rotary, device):
    """cos | sin of position * 10000^(-2 i / rotary), float32 [positions, rotary]."""
    i = torch.arange(rotary // 2, dtype=torch.float64, device=device)
    at = torch.arange(positions, dtype=torch.float64, device=device)
    a = at[:, None] * torch.exp(i * (-2.0 * math.log(10000.0) / rotary))
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    dt = DTYPE[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    if case["op"] == "norm":
        B, N = case["sequences"], case["tokens"]
        state = {"case": case, "rope": _angles(N, case["rotary"], dev),
                 "wq": 1 + 0.1 * normal(D, dtype=torch.float32),
                 "wk": 1 + 0.1 * normal(D, dtype=torch.float32)}
        for x in ("", "t", "g") + (("gt",) if case["tangents"] else ()):
            if x != "t" or case["tangents"]:
                state[x + "q"], state[x + "k"] = normal(B, H, N, D), normal(B, Hk, N, D)
        return state
    page = case["page"]
    new, past = _lengths(case)
    B, T = len(new), sum(new)
    total = [n + p for n, p in zip(new, past)]
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new).cumsum(0)
    state = {"case": case, "cu": cu.to(dev), "longest_new": max(new), "longest": max(total),
             "row_of": torch.cat([torch.arange(n) for n in new]).to(dev),
             "sequence_of": torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(dev),
             "start": torch.tensor(past, dtype=torch.int32, device=dev),
             "lens": torch.tensor(total, dtype=torch.int32, device=dev), "ks": None, "vs": None}
    # pages in no order; entries behind a sequence's last page are -1
    need = [-(-x // page) for x in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    column = torch.arange(max(need), device=dev)
    before = torch.tensor([0] + need[:-1]).cumsum(0).to(dev)
    entry = before[:, None] + column
    state["table"] = torch.where(column < torch.tensor(need, device=dev)[:, None],
                                 order[entry.clamp(max=pages - 1)], -1).to(torch.int32)
    shape = (pages, Hk, page, D)
    state["q"] = normal(T, H, D)
    if case["op"] == "append":
        state.update(k=normal(T, Hk, D), v=normal(T, Hk, D), kc=torch.zeros(shape, device=dev, dtype=dt),
                     vc=torch.zeros(shape, device=dev, dtype=dt),
                     rope=_angles(max(total), case["rotary"], dev), wq=None, wk=None)
        if case["norm"]:
            state.update(wq=1 + 0.1 * normal(D, dtype=torch.float32),
                         wk=1 + 0.1 * normal(D, dtype=torch.float32))
        return state
    kc, vc = normal(*shape), normal(*shape)
    if case["cache"] == "e4m3":
        (kc, state["ks"]), (vc, state["vs"]) = _quantise(kc), _quantise(vc)
    state.update(kc=kc, vc=vc)
    return state


def _values(codes, scale):
    """What a cache holds: its entries, times their scale where there is one."""
    x = codes.float()
    return x if scale is None else torch.ldexp(x, scale.int().unsqueeze(-1) - 127)


def _softmax(s, v):
    """Weighted averages of v and log-sum-exps for logits that may be -inf; empty rows give 0, -inf."""
    m = s.amax(-1, keepdim=True)
    s.sub_(m.clamp(min=-3e38)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v) / total.masked_fill(total == 0, 1.0)
    return o, (m + total.log()).squeeze(-1)


def _plain_chunk(st):
    case, N, M, cu = st["case"], st["longest"], st["longest_new"], st["cu"].long()
    T, H, D = st["q"].shape
    _, Hk, page, _ = st["kc"].shape
    B = len(cu) - 1
    place, token = (torch.arange(x, device=cu.device) for x in (N, M))
    table = st["table"].clamp(min=0).long()

    def dense(cache, scale):
        x = _values(cache[table], None if scale is None else scale[table])
        return x.transpose(1, 2).reshape(B, Hk, 1, -1, D)[:, :, :, :N]

    q = st["q"].float()[(cu[:-1, None] + token).clamp_(max=T - 1)]  # padded to the longest
    q = q.view(B, M, Hk, H // Hk, D).permute(0, 2, 3, 1, 4)
    position = (st["start"].long()[:, None] + token)[:, :, None]
    keep = place <= position
    if case["window"]:
        keep &= (place > position - case["window"]) | (place < case["sinks"])
    s = torch.matmul(q * (1.0 / math.sqrt(D)), dense(st["kc"], st["ks"]).transpose(-1, -2))
    s.masked_fill_(~keep[:, None, None], -math.inf)
    o, lse = _softmax(s, dense(st["vc"], st["vs"]))
    b, i = st["sequence_of"], st["row_of"]
    return {"o": o[b, :, :, i].reshape(T, H, D).to(st["q"].dtype),
            "lse": lse[b, :, :, i].reshape(T, H).t().contiguous()}


def _plain_decode(st):
    case, lens = st["case"], st["lens"].long()[:, None]
    B, H, D = st["q"].shape
    _, Hk, page, _ = st["kc"].shape
    # the positions that are visible: the window's, and the sinks in front of it
    lo = (lens - case["window"]).clamp(min=0)
    width = min(case["window"], st["longest"])
    position = torch.cat(((lo + torch.arange(width, device=lens.device)),
                          torch.arange(case["sinks"], device=lens.device).expand(B, -1)), 1)
    keep = torch.cat((position[:, :width] < lens, position[:, width:] < lo), 1)
    position = position.clamp(max=st["longest"] - 1)
    at = st["table"].gather(1, position // page).clamp(min=0).long()

    def rows(cache, scale):
        x = _values(cache[at, :, position % page],
                    None if scale is None else scale[at, :, position % page])
        return x.transpose(1, 2)

    s = torch.matmul(st["q"].float().view(B, Hk, H // Hk, D) * (1.0 / math.sqrt(D)),
                     rows(st["kc"], st["ks"]).transpose(-1, -2))
    s.masked_fill_(~keep[:, None, None], -math.inf)
    o, lse = _softmax(s, rows(st["vc"], st["vs"]))
    return {"o": o.reshape(B, H, D).to(st["q"].dtype), "lse": lse.reshape(B, H)}


def _rotate(x, rope, interleaved, back=False):
    """Pairs of the first columns of x by the angles rope = cos | sin (back: by minus them)."""
    half = rope.shape[-1] // 2
    c, s = rope[..., :half], rope[..., half:]
    if back:
        s = -s
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((turned, rest), -1)


def _plain_append(st):
    case, page = st["case"], st["kc"].shape[2]
    position = st["start"].long()[st["sequence_of"]] + st["row_of"]
    rope = st["rope"][position][:, None]
    at, place = st["table"][st["sequence_of"], position // page].long(), position % page

    def turned(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
        return _rotate(y, rope, case["interleaved"]).to(x.dtype)

    st["kc"][at, :, place] = turned(st["k"], st["wk"])
    st["vc"][at, :, place] = st["v"]
    return {"q": turned(st["q"], st["wq"]), "kc": st["kc"], "vc": st["vc"]}


def _plain_norm(st):
    case, out = st["case"], {}

    def side(x):
        w, dt = st["w" + x], st[x].dtype
        xs = st[x].float()
        r = torch.rsqrt((xs * xs).mean(-1, keepdim=True) + EPS)
        n = r * xs
        out[x] = _rotate(w * n, st["rope"], case["interleaved"]).to(dt)
        a = _rotate(st["g" + x].float(), st["rope"], case["interleaved"], back=True)
        u = w * a
        gx = r * (u - n * (n * u).mean(-1, keepdim=True))
        gw = a * n
        if case["tangents"]:
            t = st["t" + x].float()
            m = (n * t).mean(-1, keepdim=True)
            dn = r * (t - n * m)
            out["t" + x] = _rotate(w * dn, st["rope"], case["interleaved"]).to(dt)
            b = _rotate(st["gt" + x].float(), st["rope"], case["interleaved"], back=True)
            v = w * b
            p, q = (v * t).mean(-1, keepdim=True), (v * n).mean(-1, keepdim=True)
            gx = gx + r * r * (n * (3 * m * q - p) - q * t - m * v)
            gw = gw + b * dn
            out["gt" + x] = (r * (v - n * q)).to(dt)
        out["g" + x] = gx.to(dt)
        out["gw" + x] = gw.sum((0, 1, 2))

    side("q")
    side("k")
    return out


def _own(st):
    from forward_mode_flash_gb300 import api

    case = st["case"]
    if case["op"] == "chunk":
        o, lse = api.attention_chunk(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["cu"],
                                     window=case["window"] or None, sinks=case["sinks"],
                                     k_scale=st["ks"], v_scale=st["vs"], return_lse=True)
        return {"o": o, "lse": lse}
    if case["op"] == "decode":
        o, lse = api.attention_decode(st["q"], st["kc"], st["vc"], st["table"], st["lens"],
                                      window=case["window"], sinks=case["sinks"],
                                      k_scale=st["ks"], v_scale=st["vs"], return_lse=True)
        return {"o": o, "lse": lse}
    options = {"q_weight": st["wq"], "k_weight": st["wk"], "eps": EPS,
               "interleaved": case["interleaved"]}
    if case["op"] == "append":
        q = api.cache_append(st["q"], st["k"], st["v"], st["kc"], st["vc"], st["table"], st["rope"],
                             st["start"], st["cu"], **options)
        return {"q": q, "kc": st["kc"], "vc": st["vc"]}
    if not case["tangents"]:
        q, k = api.norm_rope(st["q"], st["k"], st["rope"], **options)
        gq, gk, gwq, gwk = api.norm_rope_bwd(st["q"], st["k"], st["gq"], st["gk"], st["rope"],
                                             **options)
        return {"q": q, "k": k, "gq": gq, "gk": gk, "gwq": gwq, "gwk": gwk}
    q, k, tq, tk = api.norm_rope_dual(st["q"], st["k"], st["tq"], st["tk"], st["rope"], **options)
    gq, gk, gtq, gtk, gwq, gwk = api.norm_rope_bwd_dual(
        st["q"], st["k"], st["tq"], st["tk"], st["gq"], st["gk"], st["gtq"], st["gtk"], st["rope"],
        **options)
    return {"q": q, "k": k, "tq": tq, "tk": tk, "gq": gq, "gk": gk, "gtq": gtq, "gtk": gtk,
            "gwq": gwq, "gwk": gwk}


def run(state):
    if own:
        return _own(state)
    return {"chunk": _plain_chunk, "decode": _plain_decode, "append": _plain_append,
            "norm": _plain_norm}[state["case"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits
def _rows_64(st, cache, scale, b, n, head):
    """One head's first n cached rows of a sequence, as values."""
    page, position = cache.shape[2], torch.arange(n, device=cache.device)
    at = st["table"][b].long()[position // page]
    x = cache[at, head, position % page].double()
    if scale is not None:
        x = x * torch.exp2(scale[at, head, position % page].double() - 127)[:, None]
    return x


def _attention_64(st, case):
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    new, past = _lengths(case)
    dev = st["q"].device
    o = torch.zeros(sum(new), H, D, dtype=torch.float64, device=dev)
    lse = torch.zeros(sum(new), H, dtype=torch.float64, device=dev)
    first = 0
    for b, (n, p) in enumerate(zip(new, past)):
        for hk in range(Hk if n else 0):
            k = _rows_64(st, st["kc"], st["ks"], b, n + p, hk)
            v = _rows_64(st, st["vc"], st["vs"], b, n + p, hk)
            j = torch.arange(n + p, device=dev)
            for h in range(hk * (H // Hk), (hk + 1) * (H // Hk)):
                for r in range(0, n, 2048):
                    at = slice(first + r, first + min(n, r + 2048))
                    i = p + torch.arange(r, min(n, r + 2048), device=dev)[:, None]
                    hidden = j > i
                    if case["window"]:
                        hidden = hidden | ((i - j >= case["window"]) & (j >= case["sinks"]))
                    logits = (st["q"][at, h].double() @ k.T / math.sqrt(D)).masked_fill_(
                        hidden, -math.inf)
                    z = torch.logsumexp(logits, 1)
                    o[at, h], lse[at, h] = (logits - z[:, None]).exp() @ v, z
        first += n
    return {"o": o, "lse": lse if case["op"] == "decode" else lse.t().contiguous()}


def _turn_64(x, w, rope, interleaved):
    """Norm and rotation of one row set through complex numbers."""
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    half = rope.shape[-1] // 2
    unit = torch.complex(rope[..., :half], rope[..., half:])
    if interleaved:
        y = torch.view_as_real(torch.view_as_complex(
            x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * unit).flatten(-2)
    else:
        y = torch.complex(x[..., :half], x[..., half:2 * half]) * unit
        y = torch.cat((y.real, y.imag), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("chunk", "decode"):
        return _attention_64(st, case)
    rope = st["rope"].double()
    if case["op"] == "append":
        new, past = _lengths(case)
        out, first = {"kc": st["kc"].double(), "vc": st["vc"].double()}, 0
        q = torch.zeros(st["q"].shape, dtype=torch.float64, device=rope.device)
        for b, (n, p) in enumerate(zip(new, past)):
            rows = slice(first, first + n)
            position = p + torch.arange(n, device=rope.device)
            at, place = st["table"][b].long()[position // case["page"]], position % case["page"]
            turn = rope[position][:, None]
            q[rows], k = (_turn_64(st[x][rows].double(), None if st["w" + x] is None else
                                   st["w" + x].double(), turn, case["interleaved"])
                          for x in ("q", "k"))
            out["kc"][at, :, place], out["vc"][at, :, place] = k, st["v"][rows].double()
            first += n
        return {"q": q, **out}
    out = {}
    for x in ("q", "k"):
        a, w = st[x].double().requires_grad_(), st["w" + x].double().requires_grad_()
        turn = lambda y: _turn_64(y, w, rope, case["interleaved"])  # noqa: E731
        y, wanted = turn(a), [a, w]
        loss = (y * st["g" + x].double()).sum()
        if case["tangents"]:
            # the tangent as a derivative of <y, z> with respect to a and z in turn
            t = st["t" + x].double().requires_grad_()
            z = torch.zeros_like(y).requires_grad_()
            back, = torch.autograd.grad((y * z).sum(), a, create_graph=True)
            dy, = torch.autograd.grad((back * t).sum(), z, create_graph=True)
            loss, wanted = loss + (dy * st["gt" + x].double()).sum(), wanted + [t]
            out["t" + x] = dy.detach()
        grads = torch.autograd.grad(loss, wanted)
        out[x], out["g" + x], out["gw" + x] = y.detach(), grads[0], grads[1]
        if case["tangents"]:
            out["gt" + x] = grads[2]
    return out
