"""The 8-bit cache in fp64 numpy: block scales, codes as the numbers that they are, appends block by block,
and attention token by token."""

import numpy as np

TILE = 32
D = 128


def round_e4m3(y):
    """Nearest e4m3 number (3 mantissa bits, exponents -6 .. 8, subnormal steps of 2^-9, largest 448), ties to
    the even step; saturating."""
    a = np.minimum(np.abs(y), 448.0)
    with np.errstate(divide="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(e - 3)
    return np.sign(y) * np.minimum(np.round(a / step) * step, 448.0)


def round_s8(y):
    return np.clip(np.round(y), -127.0, 127.0)


def block_scale(amax, code):
    """The scale that a block of largest finite magnitude amax asks for."""
    if code == "e4m3":
        e = -100
        while 448.0 * 2.0 ** e < amax and e < 120:
            e += 1
        return 2.0 ** e
    s = max(amax / 127.0, 2.0 ** -100)
    step = 2.0 ** (np.floor(np.log2(s)) - 7)
    return float(np.ceil(s / step) * step)


class Cache8:
    """Codes [batch][Hkv][capacity][128] (NaN: nothing there) and scales [batch][Hkv][capacity/32] of K and V."""

    def __init__(self, batch, n_kv_heads, capacity, code):
        self.code = code
        self.cap = capacity
        self.codes = np.full((2, batch, n_kv_heads, capacity, D), np.nan)
        self.scales = np.full((2, batch, n_kv_heads, capacity // TILE), np.nan)

    def append(self, side, b, x, start):
        """x: [n][Hkv][128] at positions start ..; positions outside [0, capacity) are left out."""
        rnd = round_e4m3 if self.code == "e4m3" else round_s8
        x = np.asarray(x, dtype=np.float64)
        for h in range(x.shape[1]):
            for t in range(self.cap // TILE):
                pos = [p for p in range(TILE * t, TILE * t + TILE) if start <= p < start + x.shape[0]]
                if not pos:
                    continue
                y = np.where(np.isnan(x[pos[0] - start: pos[-1] - start + 1, h]), 0.0,
                             x[pos[0] - start: pos[-1] - start + 1, h])
                fin = np.abs(y[np.isfinite(y)])
                now = block_scale(fin.max() if fin.size else 0.0, self.code)
                old = slice(TILE * t, pos[0])
                if pos[0] > TILE * t:
                    was = self.scales[side, b, h, t]
                    if now > was:
                        self.codes[side, b, h, old] = rnd(self.codes[side, b, h, old] * was / now)
                    else:
                        now = was
                self.scales[side, b, h, t] = now
                self.codes[side, b, h, pos] = rnd(np.clip(y, -1e39, 1e39) / now)

    def values(self, side, b, h, n):
        return self.codes[side, b, h, :n] * np.repeat(self.scales[side, b, h], TILE)[:n, None]


def attention(q, k, v, scale):
    """q: [Hq][128] rows over k, v: [Hkv][T][128]; rows of zeros where T is 0."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    out = np.zeros_like(q)
    g = q.shape[0] // k.shape[0]
    if k.shape[1] == 0:
        return out
    for i in range(q.shape[0]):
        s = k[i // g] @ q[i] * scale
        p = np.exp(s - s.max())
        out[i] = (p / p.sum()) @ v[i // g]
    return out
