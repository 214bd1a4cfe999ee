"""Plain float64 definitions of the packed-prompt and paged-cache operators,
and the error bounds their tests use.

Bounds (u = half a unit in the last place of the tensors' type, finfo.eps / 2;
w = that of the weights' type in the matrix product, 0 on the CUDA cores):
an output is the average sum_j p_j v_j with
  - each weight off by a relative w (its rounding), 2 ds (an error ds of the
    logits changes exp by e^ds - 1 <= 2 ds for ds <= 1) and 2^-20 (the
    exponential and the rescaling steps), numerator and denominator alike,
    which moves the average by at most twice that times sum_j p_j |v_j|;
  - n + 8 roundings of fp32 accumulation, 2^-24 each, in numerator and
    denominator;
  - one rounding u of the result.
ds = (D + 8) 2^-24 scale max_j sum_d |q_d k_jd|: D products and sums in fp32
and a few for the scaling.  The tensor cores may truncate instead of round in
their sums, so every fp32 step counts 2^-23 there.
"""

import math

import numpy as np


def f64(t):
    import torch
    return t.detach().to("cpu", torch.float64).numpy()


def attend(q, k, v, keep, scale):
    """Float64 attention of rows q [M, D] on k, v [N, D] over keep [M, N].

    Returns o, lse, average |v| (sum_j p_j |v_j|) and the largest
    scale * sum_d |q_d k_d| over each row's kept keys."""
    M, N = keep.shape
    o, lse = np.zeros((M, v.shape[1])), np.full(M, -np.inf)
    mag, big = np.zeros_like(o), np.zeros(M)
    if N == 0:
        return o, lse, mag, big
    with np.errstate(all="ignore"):
        s = np.where(keep, q @ k.T * scale, -np.inf)
        big = np.where(keep, np.abs(q) @ np.abs(k).T * abs(scale), 0.0).max(1)
        m = s.max(1, keepdims=True)
        e = np.exp(s - np.where(np.isneginf(m), 0.0, m))
        tot = e.sum(1, keepdims=True)
    some = keep.any(1)
    vz = np.where(keep.any(0)[:, None], v, 0.0)  # rows no query keeps have no say
    p = e[some] / tot[some]
    o[some], mag[some] = p @ vz, p @ np.abs(vz)
    lse[some] = (m + np.log(tot))[some, 0]
    return o, lse, mag, big


def bounds(o, lse, mag, big, n, D, u, w, tensor_cores):
    """Largest allowed errors of o and lse (see the module's docstring)."""
    step = 2.0 ** -23 if tensor_cores else 2.0 ** -24
    ds = (D + 8) * step * big
    rel = w + 2 * ds + 2.0 ** -20 + (n + 8) * step
    tiny = 2.0 ** -24 if w else 2.0 ** -126  # fp16's smallest step: results near zero
    b_o = u * np.abs(o) + 2 * rel[:, None] * mag + tiny
    fin = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    b_lse = ds + 2.0 ** -20 + (n + 8) * step + 4 * 2.0 ** -24 * (fin + big)
    return b_o, b_lse


def quantise(x):
    """(codes as values, exponents) of rows x [..., D]: the definition."""
    top = np.nanmax(np.where(np.isnan(x), 0.0, np.abs(x)), axis=-1)
    e = np.full(top.shape, -127, dtype=np.int64)
    for i, t in np.ndenumerate(top):
        if np.isinf(t):
            e[i] = 120
        elif t > 0:
            _, p = math.frexp(t)           # t = f 2^p, 0.5 <= f < 1
            k = p - 9                      # 448 2^k = 0.875 2^p
            e[i] = max(-127, k if t <= 448 * 2.0 ** k else k + 1)
    y = x / np.exp2(e.astype(np.float64))[..., None]
    return round_e4m3(y), e


def round_e4m3(y):
    """Nearest e4m3 value, ties to even; saturating at 448, NaN kept."""
    with np.errstate(all="ignore"):
        mag = np.clip(np.abs(y), 2.0 ** -20, 448.0)
        step = np.exp2(np.maximum(np.floor(np.log2(mag)), -6) - 3)
        r = np.rint(np.clip(y, -448.0, 448.0) / step) * step
    return np.where(np.isnan(y), np.nan, r)


class Cache:
    """A paged cache with random page placement, on the CPU (made there)."""

    def __init__(self, lens, Hkv, D, page, dtype, e4m3, seed, spare=2, extra_cols=1):
        import torch
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(need + [0]) + extra_cols), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.lens, self.page, self.Hkv, self.D = list(lens), page, Hkv, D
        self.dtype, self.e4m3 = dtype, e4m3
        shape = (self.pages, Hkv, page, D)
        self.scales = None
        kv = [torch.randn(shape, generator=g) for _ in range(2)]
        if e4m3:
            # a spread of magnitudes over rows, so that scales matter
            kv = [x * torch.exp2(torch.randint(-6, 7, shape[:3], generator=g).float())[..., None] * 0.25
                  for x in kv]
            q = [quantise(x.double().numpy()) for x in kv]
            self.k, self.v = (torch.from_numpy(c).to(torch.float8_e4m3fn) for c, _ in q)
            self.scales = [torch.from_numpy(e + 127).to(torch.uint8) for _, e in q]
        else:
            self.k, self.v = (x.to(dtype) for x in kv)

    def rows(self, b, n=None):
        """Float64 keys and values [Hkv, n, D] of a sequence's first n positions."""
        n = self.lens[b] if n is None else n
        pos = np.arange(n)
        pg, r = self.table[b].numpy()[pos // self.page], pos % self.page
        out = []
        for i, c in enumerate((self.k, self.v)):
            x = c.double().numpy()[pg, :, r]
            if self.e4m3:
                s = self.scales[i].numpy()[pg, :, r].astype(np.float64)
                x = x * np.exp2(s - 127)[..., None]
            out.append(x.transpose(1, 0, 2))
        return out

    def cuda(self):
        return dict(k_cache=self.k.cuda(), v_cache=self.v.cuda(), block_table=self.table.cuda(),
                    k_scale=self.scales[0].cuda() if self.e4m3 else None,
                    v_scale=self.scales[1].cuda() if self.e4m3 else None)
