"""Rotary positions in fp64 numpy: frequencies by their definitions, pairs as complex numbers."""

import math

import numpy as np


def frequencies(rotary_dim, base, scaling="plain", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    half = rotary_dim // 2
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = np.array([base ** (-2.0 * i / rotary_dim) for i in range(half)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "bands":
        out = []
        for x in f:
            turns = original_len / (2 * math.pi / x)
            if turns >= high:
                out.append(x)
            elif turns <= low:
                out.append(x / factor)
            else:
                s = (turns - low) / (high - low)
                out.append((1 - s) * x / factor + s * x)
        return np.array(out), 1.0
    if scaling == "yarn":
        def index(turns):
            return rotary_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rotary_dim - 1)
        if hi <= lo:
            hi = lo + 0.001
        ramp = np.clip((np.arange(half) - lo) / (hi - lo), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, pos, freq, layout, mscale=1.0, inverse=False):
    """x: [n][heads][128]; pos: [n]."""
    x = np.asarray(x, dtype=np.float64)
    rd = 2 * len(freq)
    ang = np.remainder(np.asarray(pos, dtype=np.float64)[:, None] * freq, 2 * math.pi)
    w = (mscale * np.exp((-1j if inverse else 1j) * ang))[:, None]
    out = x.copy()
    if layout == "half":
        z = (x[..., : rd // 2] + 1j * x[..., rd // 2: rd]) * w
        out[..., : rd // 2], out[..., rd // 2: rd] = z.real, z.imag
    else:
        z = (x[..., 0:rd:2] + 1j * x[..., 1:rd:2]) * w
        out[..., 0:rd:2], out[..., 1:rd:2] = z.real, z.imag
    return out
