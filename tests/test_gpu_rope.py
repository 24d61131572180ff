"""Rotary positions on the GPU against the fp64 oracle.

Tolerance per value, r = mscale * hypot(x0, x1) the length of its pair and u = 2^-24: the angle is off by 2^-23 of a
turn's fraction and rounding (at most 4e-7 rad with the position's double product), sine and cosine by 2 u, products
and sum by 3 u: r * 1e-6; and half a step of the output type."""

import numpy as np
import pytest
import torch

from oracle import rope
from rotated_bit_kv_iq_b200 import binding as B
from tests._helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_bit_kv_iq_b200 import build

    build.build()
    B.lib()


def _check(got, x, pos, freq, layout, ms, inverse, dtype):
    x = x.double().cpu().numpy()
    want = rope.rotate(x, pos, freq, layout, ms, inverse)
    rd = 2 * len(freq)
    got = got.double().cpu().numpy()
    np.testing.assert_array_equal(got[..., rd:], x[..., rd:])
    half = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}[dtype]
    top = np.abs(x).max() * 1.5 * abs(ms)
    tol = np.abs(want) * half + top * 1e-6 + (2.0 ** -25 if dtype == F16 else 0)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rd", [128, 64, 112, 2, 74, 8])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_the_oracle(dtype, layout, rd, inverse):
    freq, ms = B.iq_rope_frequencies(rd, 10000.0, "yarn" if rd > 2 else "plain", 8.0, 4096.0)
    f = torch.from_numpy(freq).to(DEV)
    g = torch.Generator().manual_seed(rd)
    for n, hq, hk in ((1, 1, 1), (5, 12, 2), (33, 7, 7)):
        pos = [int(p) for p in torch.randint(-5, 1 << 17, (n,), generator=g)]
        pos[0] = 2 ** 31 - 1
        q, k = (torch.randn((n, h, 128), generator=g).to(dtype).to(DEV) for h in (hq, hk))
        qo, ko = Guarded(q.shape, dtype, fill=9.0), Guarded(k.shape, dtype, fill=9.0)
        p = torch.tensor(pos, dtype=torch.int32, device=DEV)
        B.iq_rope(q, k, p, f, qo.t, ko.t, layout, ms, inverse)
        torch.cuda.synchronize()
        qo.check("q_out")
        ko.check("k_out")
        _check(qo.t, q, pos, freq, layout, ms, inverse, dtype)
        _check(ko.t, k, pos, freq, layout, ms, inverse, dtype)
        # in place the same bits, and one side alone
        want = qo.t.clone()
        B.iq_rope(q, None, p, f, layout=layout, mscale=ms, inverse=inverse)
        assert torch.equal(q, want)
        B.iq_rope(None, k, p, f, None, ko.t, layout, ms, inverse)
        B.iq_rope(None, k, p, f, layout=layout, mscale=ms, inverse=inverse)
        assert torch.equal(k, ko.t)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rd", [128, 40, 10])
def test_rope_slices_of_a_fused_projection(layout, rd):
    freq, _ = B.iq_rope_frequencies(rd)
    f = torch.from_numpy(freq).to(DEV)
    qkv = torch.randn((17, 12, 128), generator=torch.Generator().manual_seed(2)).to(F16).to(DEV)
    keep = qkv.clone()
    pos = list(range(1000, 1017))
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)
    B.iq_rope(qkv[:, :8], qkv[:, 8:10], p, f, layout=layout)  # in place
    _check(qkv[:, :8], keep[:, :8], pos, freq, layout, 1.0, False, F16)
    _check(qkv[:, 8:10], keep[:, 8:10], pos, freq, layout, 1.0, False, F16)
    assert torch.equal(qkv[:, 10:], keep[:, 10:])


def test_rope_inverse_is_the_gradient():
    """d/dx <w, rope(x)> = rope^-1(w) (times mscale), against the formula and against differences in float32."""
    freq, ms = B.iq_rope_frequencies(96, 10000.0, "yarn", 4.0, 2048.0)
    f = torch.from_numpy(freq).to(DEV)
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randn((3, 2, 128), generator=g).to(DEV) for _ in range(2))
    p = torch.tensor([0, 77, 4000], dtype=torch.int32, device=DEV)
    grad = torch.empty_like(w)
    B.iq_rope(w, None, p, f, grad, mscale=ms, inverse=True)
    _check(grad, w, p.tolist(), freq, "half", ms, True, F32)
    y = torch.empty_like(x)
    for idx in ((0, 0, 3), (1, 1, 50), (2, 0, 94), (2, 1, 100)):
        d = []
        for s in (1.0, -1.0):
            z = x.clone()
            z[idx] += s * 0.5
            B.iq_rope(z, None, p, f, y, mscale=ms)
            d.append((y.double() * w.double()).sum().item())
        # the map is linear: only the roundings of 256 terms of two sums are left
        assert abs(d[0] - d[1] - grad[idx].item()) < 1e-4


def test_rope_on_another_stream_and_in_a_graph():
    freq, _ = B.iq_rope_frequencies(128)
    f = torch.from_numpy(freq).to(DEV)
    q = torch.randn((4, 8, 128), generator=torch.Generator().manual_seed(5)).to(BF16).to(DEV)
    p = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device=DEV)
    o = torch.empty_like(q)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.iq_rope(q, None, p, f, o)
        p.add_(1)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    _check(o, q, [3, 4, 5, 6], freq, "half", 1.0, False, BF16)
