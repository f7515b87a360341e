"""Paged caches for the cache operators' tests and their attention in float64.

A Pool builds page pools (bf16 or 4-bit) from float32 rows with numpy; every
byte that no cached position owns is 0xFF (NaN in every format), so a kernel
that lets an unseen position into a sum shows it.
"""
import numpy as np

from synth import f32_to_bf16_bits

PAGE = 32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def e4m3_values():
    """The value of every e4m3 byte (NaN at 0x7F and 0xFF)."""
    b = np.arange(256)
    e, m = b >> 3 & 15, b & 7
    v = np.where(e == 0, m / 512.0, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b & 128, -v, v)


def quantise(x):
    """float32 rows [..., D] -> codes [..., D], block scales [..., D/16], row scales [...], one float32 operation
    per step; a row with an infinity or a NaN has the row scale NaN and zeros elsewhere."""
    x = np.asarray(x, np.float32)
    f = np.float32
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(x).all(-1)
        s = np.where(bad, f(np.nan), (np.abs(x).max(-1) / f(2688)).astype(f))
        s6 = (s * f(6))[..., None]
        want = np.minimum((np.abs(blocks).max(-1) / s6).astype(f), f(448))
        want = np.where(s6 > 0, want, f(0)).astype(np.float64)
        # e4m3, round to nearest even: a step of 2^(e-3), 2^-9 below 2^-6
        ulp = 2.0 ** (np.floor(np.log2(np.maximum(want, 2.0 ** -6))) - 3)
        b = np.rint(want / ulp) * ulp
        step = (b.astype(f) * s[..., None]).astype(f)[..., None]
        r = np.where(step > 0, np.clip((blocks / step).astype(f), f(-6), f(6)), f(0)).astype(np.float64)
        ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(r), 1.0))) - 1)
        v = np.rint(r / ulp) * ulp
    codes = np.searchsorted(E2M1, np.abs(v)).astype(np.uint8) | ((r < 0).astype(np.uint8) << 3)
    sb = np.searchsorted(e4m3_values()[:127], b).astype(np.uint8)
    return codes.reshape(x.shape), sb, s.astype(f)


def dequantise(codes, sb, s):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    v = v.reshape(*v.shape[:-1], v.shape[-1] // 16, 16) * e4m3_values()[sb][..., None]
    return v.reshape(codes.shape) * s[..., None].astype(np.float64)


def v_byte(r, d, D):
    return ((r >> 1 & 3) * (D // 16) + d // 16) * 64 + (r >> 3) * 16 + d % 16


def head_bytes(fmt, D):
    return PAGE * D * 2 if fmt == "bf16" else PAGE * (D // 2 + D // 16 + 4)


class Pool:
    """K and V pools of `lens` cached positions per sequence, pages in a random order."""

    def __init__(self, fmt, Hkv, D, lens, seed, stride=None, spare=2, scale=1.0):
        self.fmt, self.Hkv, self.D, self.lens = fmt, Hkv, D, list(lens)
        rng = np.random.default_rng(seed)
        need = [(n + PAGE - 1) // PAGE for n in lens]
        self.stride = stride or max(1, max(need))
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(lens), self.stride), -1, np.int32)   # unused entries: not a page
        self.k, self.v = [], []          # values held, float64 [n, Hkv, D]
        self.K = np.full((self.n_pages, Hkv, head_bytes(fmt, D)), 0xFF, np.uint8)
        self.V = self.K.copy()
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            ch = np.exp(0.5 * rng.standard_normal((2, 1, Hkv, D)))
            for isv, keep in ((0, self.k), (1, self.v)):
                x = (rng.standard_normal((n, Hkv, D)) * ch[isv] * scale).astype(np.float32)
                keep.append(self.put(isv, b, 0, x))

    def put(self, isv, b, first, x):
        """Stores float32 rows x [n, Hkv, D] at positions first.. of sequence b; returns the values held."""
        D, pool = self.D, self.V if isv else self.K
        if self.fmt == "bf16":
            bits = f32_to_bf16_bits(x.astype(np.float32))
            held = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        else:
            codes, sb, s = quantise(x)
            held = dequantise(codes, sb, s)
        for i in range(x.shape[0]):
            pg, r = self.table[b, (first + i) // PAGE], (first + i) % PAGE
            for g in range(self.Hkv):
                head = pool[pg, g]
                if self.fmt == "bf16":
                    head.view(np.uint16)[r * D:(r + 1) * D] = bits[i, g]
                    continue
                c, d = codes[i, g], np.arange(D)
                if isv:
                    at = v_byte(r, d, D)
                    head[at] = (head[at] & 0xF0 | c) if r % 2 == 0 else (head[at] & 0x0F | c << 4)
                    head[PAGE * D // 2 + np.arange(D // 16) * PAGE + r] = sb[i, g]
                else:
                    head[r * D // 2:(r + 1) * D // 2] = c[0::2] | c[1::2] << 4
                    head[PAGE * D // 2 + r * D // 16:PAGE * D // 2 + (r + 1) * D // 16] = sb[i, g]
                head[PAGE * (D // 2 + D // 16):].view(np.float32)[r] = s[i, g]
        return held


def attention(q, k, v, n, window=0, sinks=0, scale=None, hidden=None):
    """q float64 [r, Hq, D], the last r of n positions; k, v float64 [n, Hkv, D] -> out, sum p|v| (the same shape),
    per (row, head) the largest scale * sum |q||k| over what the row sees, and the largest p_j max|v_j|."""
    r, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = scale or D ** -0.5
    out, mass, reach, peak = np.zeros_like(q), np.zeros_like(q), np.zeros((r, Hq)), np.zeros((r, Hq))
    p, j = np.arange(n - r, n)[:, None], np.arange(n)[None]
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    if hidden is not None:
        see &= ~hidden
    rows = see.any(1)
    used = see.any(0)                       # what no row sees may be anything
    for h in range(Hq):
        kg, vg = (np.where(used[:, None], x[:n, h // G], 0.0) for x in (k, v))
        z = np.where(see, (q[:, h] @ kg.T) * scale, -np.inf)
        top = np.where(rows, z.max(1, initial=-np.inf), 0.0)
        w = np.exp(z - top[:, None])
        w /= np.where(rows, w.sum(1), 1.0)[:, None]
        out[:, h], mass[:, h] = w @ vg, w @ np.abs(vg)
        reach[:, h] = np.where(see, np.abs(q[:, h]) @ np.abs(kg).T, 0.0).max(1, initial=0.0) * scale
        peak[:, h] = (w * np.abs(vg).max(1, initial=0.0)[None]).max(1, initial=0.0)
    return out, mass, reach, peak


def tolerance(out, mass, reach, peak, D, n, dtype, fmt):
    """How far an output may be.  A score is a float32 sum of D products of exact keys with queries of 22 or more
    bits: off by at most d = (D + 8) 2^-24 reach (+ 2^-22 reach for the queries' bits).  A probability's relative
    error is then 2 d plus the exponential's 2^-20; numerator and denominator each carry it and the n + 64 additions
    of a float32 sum (2^-24 each, against the sum of p|v|).  4-bit pages: a weight p * (row scale) enters as f16
    parts whose smallest step is 2^-24 where the largest weight is at least 2^7: each of n weights is off by at most
    2^-25 / 2^7 of the largest one, and its element is at most its row's largest.  bf16 rows: the probabilities'
    rounding to bf16 (half a step: 2^-8 of each) and the output's (2^-8 of it)."""
    d = ((D + 8) * 2.0 ** -24 + 2.0 ** -22) * reach[..., None]
    t = (2 * (2 * d + 2.0 ** -20) + 2 * (n + 64) * 2.0 ** -24) * mass
    if fmt == "nvfp4":
        t = t + n * 2.0 ** -32 * peak[..., None]
    if dtype == "bf16":
        t = t + 2.0 ** -8 * mass + 2.0 ** -8 * (np.abs(out) + t)
    return t + 1e-30
