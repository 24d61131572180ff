"""CPU pins of the oracle's 8-bit cache, rotary positions and pages."""

import math

import numpy as np
import pytest
import torch

from oracle import cache8, pages, rope


def test_e4m3_rounding_is_torchs():
    g = np.random.default_rng(1)
    y = np.concatenate([g.standard_normal(4000) * 2.0 ** g.integers(-12, 9, 4000), np.arange(-460, 461) / 2.0,
                        np.arange(-40, 41) * 2.0 ** -10, [0.0, 448.0, 464.0, 1e9]]).astype(np.float32)
    want = torch.from_numpy(y).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(cache8.round_e4m3(y.astype(np.float64)), want)


@pytest.mark.parametrize("code", ["e4m3", "s8"])
def test_block_scale_is_the_smallest_of_its_kind(code):
    top = 448.0 if code == "e4m3" else 127.0
    for a in (0.0, 1e-40, 1.0, 447.9, 448.0, 448.1, 127.0, 127.01, 65504.0, 3e38):
        s = cache8.block_scale(a, code)
        m, e = math.frexp(s)
        assert m * 256 == int(m * 256) and (code == "s8" or m == 0.5)  # 8 significant bits, or a power of two
        assert s * top >= a and s >= 2.0 ** -100
        below = s / 2 if code == "e4m3" else s - 2.0 ** (e - 8)
        assert below * top < a or s == 2.0 ** -100


def test_a_block_that_grows_rounds_its_codes_again():
    c = cache8.Cache8(1, 1, 32, "s8")
    x = np.zeros((2, 1, 128))
    x[0, 0, :3] = (1.0, 0.3, -0.7)
    x[1, 0, 0] = 12.7
    c.append(0, 0, x[:1], 0)
    s0 = c.scales[0, 0, 0, 0]
    first = c.codes[0, 0, 0, 0].copy()
    assert first[0] == np.round(1.0 / s0) and s0 >= 1 / 127
    c.append(0, 0, x[1:], 1)
    s1 = c.scales[0, 0, 0, 0]
    assert s1 >= 0.1 and s1 < 0.1 * (1 + 2.0 ** -7)
    np.testing.assert_array_equal(c.codes[0, 0, 0, 0], np.round(first * s0 / s1))
    # tokens that fit leave the scale, and another order of the calls gives it again
    c.append(0, 0, x[:1], 2)
    assert c.scales[0, 0, 0, 0] == s1


def test_attention_is_torchs():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((6, 128)), g.standard_normal((2, 9, 128)), g.standard_normal((2, 9, 128))
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).view(2, 3, 128), torch.from_numpy(k), torch.from_numpy(v), scale=0.2)
    np.testing.assert_allclose(cache8.attention(q, k, v, 0.2), want.reshape(6, 128).numpy(), rtol=1e-12, atol=1e-13)
    assert not cache8.attention(q, k[:, :0], v[:, :0], 0.2).any()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_the_matrix_and_is_undone(layout):
    g = np.random.default_rng(3)
    x, pos = g.standard_normal((5, 2, 128)), np.array([0, 1, -3, 1000, 2 ** 31 - 1])
    f, _ = rope.frequencies(24, 10000.0)
    y = rope.rotate(x, pos, f, layout)
    for n in range(5):
        for i in range(12):
            a, b = (i, i + 12) if layout == "half" else (2 * i, 2 * i + 1)
            t = math.remainder(float(pos[n]) * f[i], 2 * math.pi)
            r = np.array([[math.cos(t), -math.sin(t)], [math.sin(t), math.cos(t)]])
            np.testing.assert_allclose(y[n][:, [a, b]], x[n][:, [a, b]] @ r.T, atol=1e-9)
    np.testing.assert_array_equal(y[..., 24:], x[..., 24:])
    np.testing.assert_allclose(rope.rotate(y, pos, f, layout, inverse=True), x, atol=1e-12)
    # scores depend on the distance alone
    q, k = x[:1].repeat(2, 0), x[1:2].repeat(2, 0)
    s = (rope.rotate(q, [7, 107], f, layout) * rope.rotate(k, [3, 103], f, layout)).sum(-1)
    np.testing.assert_allclose(s[0], s[1], rtol=1e-10)


def test_frequencies_by_their_limits():
    f, ms = rope.frequencies(128, 10000.0)
    assert f[0] == 1.0 and ms == 1.0 and abs(f[32] - 0.01) < 1e-15
    np.testing.assert_allclose(rope.frequencies(128, 1e4, "linear", 4.0)[0], f / 4)
    n, _ = rope.frequencies(128, 1e4, "ntk", 8.0)
    assert n[0] == 1.0 and abs(n[63] * 8 / f[63] - 1) < 1e-9  # the slowest pair is stretched by the factor
    for s in ("bands", "yarn"):
        g, ms = rope.frequencies(128, 1e4, s, 8.0, 8192.0, 1.0, 32.0)
        turns = 8192 * f / (2 * math.pi)
        np.testing.assert_array_equal(g[turns > 40], f[turns > 40])
        np.testing.assert_allclose(g[turns < 0.8], f[turns < 0.8] / 8, rtol=1e-12)
        assert (np.diff(g) < 0).all() and ms == (1.0 if s == "bands" else 0.1 * math.log(8) + 1)


def test_pages_by_hand():
    pool = np.arange(6)[None, :, None, None, None] * np.ones((1, 6, 1, 2, 1))
    t = pages.Pages(4, 3, 64, 6, [pool])
    t.extend([2, 0], [65, 10])
    assert t.table[2] == [0, 1, -1] and t.table[0] == [2, -1, -1] and t.ref == [1, 1, 1, 0, 0, 0]
    t.fork([2, 2], [1, 3])
    assert t.table[1] == [0, 3, -1] and t.table[3] == [0, 4, -1] and t.ref == [3, 1, 1, 1, 1, 0]
    assert pool[0, :, 0, 0, 0].tolist() == [0, 1, 2, 1, 1, 5] and pool[0, 3, 0, 1, 0] == 3  # one tile of two in use
    t.free([2, 0])
    assert t.ref == [2, 0, 0, 1, 1, 0] and t.table[2] == [-1] * 3 and t.status == 0
    assert t.compact() == 3
    assert t.table[1] == [0, 1, -1] and t.table[3] == [0, 2, -1] and t.ref == [2, 1, 1, 0, 0, 0]
    t.extend([0, 0, 2], [1, 1, 193])
    assert t.status == pages.SEQ | pages.NOPAGE and t.len == [1, 65, 0, 65]
    t.copy([0, 1, 9], [5, 5, 0])
    assert t.status & pages.PAGE and pool[0, 5, 0, 0, 0] == 0
