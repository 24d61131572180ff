"""The 8-bit cache on the GPU at the ends of its types: infinities beside the largest numbers, records in which nothing was
written, queries near float32's largest number, values of very different size, and batches most of whose blocks are empty.
Tolerances of attention as in tests/test_gpu_cache8.py unless a test says otherwise."""

import numpy as np
import pytest
import torch

from oracle import cache8
from rotated_bit_kv_iq_b200 import binding as B
from tests.test_gpu_cache8 import BF16, DEV, F16, F32, Held, _check_prefill, _check_rows, _decode, _filled, _i32, _prefill, _tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_bit_kv_iq_b200 import build

    build.build()
    B.lib()


def _codes(h, side, b, head, n, layer=1):
    """The first n tokens' codes as the numbers that they stand for, from the records' bytes."""
    kind = torch.float8_e4m3fn if h.code == "e4m3" else torch.int8
    tiles, out = h.c.tiles()[layer].cpu(), []
    for t in range(n):
        page = b if h.table is None else int(h.table[b, t // h.ps])
        rec, s = tiles[page, head, t % h.ps // 32], t % 32
        row = rec[4096 * side + 128 * s: 4096 * side + 128 * s + 128].view(8, 16)
        out.append(torch.cat([row[c ^ (s & 7)] for c in range(8)]).view(kind).double())
    return torch.stack(out).numpy()


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_append_infinities_beside_the_largest_numbers(code, dtype):
    """An infinity is the largest code of its sign whatever its block's scale: in one block with the type's largest numbers,
    and appended behind them."""
    big = torch.finfo(dtype).max
    h = Held(1, 1, 96, 1, code, contiguous=True)
    x = torch.zeros((1, 70, 1, 128))
    x[0, :, 0, :6] = torch.tensor([big, -big, float("inf"), float("-inf"), float("nan"), 1.0])
    x[0, 1::3, 0, 8:] = torch.tensor([float("inf"), -big, float("-inf"), big / 2, float("inf")]).repeat(24)
    x[0, 40, 0, :] = float("-inf")
    x[0, 69, 0, :] = float("inf")
    x = x.to(dtype)
    h.append(x[:, :50], -x[:, :50], [0])
    h.append(x[:, 50:], -x[:, 50:], [50])
    for side in (0, 1):
        np.testing.assert_array_equal(_codes(h, side, 0, 0, 70), h.o.codes[side, 0, 0, :70])
    assert h.c.status.item() == 0
    h.pool.check("pool")


SCALES = [float("nan"), 0.0, -1.0, float("inf"), float("-inf"), -0.0]


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("side", [0, 1])
def test_records_in_which_nothing_was_written_are_left_out(code, dtype, side):
    """A K or V scale that is no positive finite number: the record's tokens are left out and flagged, by decode and by
    prefill, whatever its codes are (here NaN ones too)."""
    lens = [300, 70, 33, 400]
    h = _filled(4, 2, 32, 13, code, lens, 70, dtype)
    bad = {0: [0, 1, 2, 3, 6, 9], 1: [0, 1, 2], 2: [1], 3: []}
    n = 0
    for b, tiles in bad.items():
        for t in tiles:
            rec = h.c.tiles()[1, int(h.table[b, t])]
            rec[:, 0, 4096 * (n % 2): 4096 * (n % 2) + 4096] = 0x7F
            at = 8192 + 4 * side
            rec[:, 0, at: at + 4] = torch.tensor([SCALES[n % len(SCALES)]]).view(torch.uint8).to(DEV)
            n += 1

    def keep(b, n):
        return np.array([p for p in range(n) if p // 32 not in bad[b]], dtype=int)

    def rows(b, n):
        kv = [h.kv(b, i, n) for i in range(2)]
        at = keep(b, n)
        return np.stack([x[0][at] for x in kv]), np.stack([x[1][at] for x in kv])

    q = torch.randn((4, 8, 128), generator=torch.Generator().manual_seed(2)).to(dtype)
    o = _decode(h, q, lens, 416)
    assert h.c.status.item() == B.IQ_DEVERR_PAGE and not o[1].any()
    for b, n in enumerate(lens):
        _check_rows(o[b], q[b].double().numpy(), *rows(b, n), 128 ** -0.5, dtype)
    h.c.status.zero_()
    start, cnt = [260, 30, 0, 360], [40, 40, 33, 40]
    q = torch.randn((4, 40, 8, 128), generator=torch.Generator().manual_seed(3)).to(dtype)
    o = _prefill(h, q, start, 416, cnt)
    assert h.c.status.item() == B.IQ_DEVERR_PAGE
    for b, s in enumerate(start):
        assert (o[b, cnt[b]:] == 7.0).all()
        for i in range(0, cnt[b], 3):
            _check_rows(o[b, i], q[b, i].double().numpy(), *rows(b, s + i + 1), 128 ** -0.5, dtype, one_term=dtype != F32)
    # behind the last token a record may hold anything
    h.c.status.zero_()
    assert not _decode(h, q[:, 0], [0, 0, 0, 0], 416).any()
    _decode(h, q[:, 0], [0, 0, 32, 0], 416)
    assert h.c.status.item() == 0


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_queries_near_the_largest_number(code, dtype):
    """Finite queries up to the type's largest number over keys so small that the scores are ordinary."""
    big = torch.finfo(dtype).max
    h = Held(2, 1, 64, 2, code)
    k = torch.zeros((2, 100, 1, 128))
    k[..., :3] = torch.randint(-8, 9, (2, 100, 1, 3), generator=torch.Generator().manual_seed(1)) * 2.0 ** -100
    v = _tokens(2, (2, 100, 1, 128), dtype)
    h.append(k.to(dtype), v, [0, 0])
    q = torch.zeros((2, 4, 128))
    q[:, 0, 0] = big
    q[:, 1, :2] = torch.tensor([2.0 ** 127, -big])
    q[:, 2, :3] = torch.tensor([-big, 2.0 ** 126, 1.0])
    q[:, 3, :2] = torch.tensor([big / 2, big])
    q = q.to(dtype)
    o = _decode(h, q, [100, 37], 128, 2.0 ** -30)
    for b, n in enumerate((100, 37)):
        kk, vv = h.kv(b, 0, n)
        _check_rows(o[b], q[b].double().numpy(), kk[None], vv[None], 2.0 ** -30, dtype)
    qq = q[:, None].repeat(1, 9, 1, 1)
    o = _prefill(h, qq, [91, 20], 128, None, 2.0 ** -30)
    _check_prefill(h, qq, o, [91, 20], [9, 9], dtype, 2.0 ** -30)
    assert h.c.status.item() == 0


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("small", [0, 2, 6])
def test_decode_small_values_beside_large_ones(code, dtype, small):
    """The block `small` of V's of 2^-12 (2^-30 in float32) has all the weight, the others, of V's of 2^12 (2^30), none: what
    comes out is the small block's, to the tolerance of the block's own values.  Per value, with w the weights and m_i =
    w_i times the largest |V| of i's block: sum w |V| (1.5 e_s + 2^-20 + T 2^-24), and, since weights times block scales are
    held in two binary16 terms of steps down to 2^-24 below their maximum (a code times scale at most twice the largest
    |V| of the block), T 2^-24 max m_i; and half a step of the output's type."""
    e, T, scale = (30, 224, 0.1) if dtype == F32 else (10, 224, 0.1)
    h = Held(1, 1, 256, 1, code, contiguous=True)
    k, v = 0.2 * _tokens(60, (1, T, 1, 128), F32), _tokens(61, (1, T, 1, 128), F32)
    q = torch.randn((1, 4, 128), generator=torch.Generator().manual_seed(3)).to(dtype)
    q[..., 9] = 30.0
    lo, hi = 32 * small, 32 * small + 32
    k[..., 9] = -60.0  # score 30 * -60 * 0.1 = -180: weight 2^-260
    k[:, lo:hi, :, 9] = 0.0
    v *= 2.0 ** e
    v[:, lo:hi] *= 2.0 ** (-2 * e)
    h.append(k, v, [0])
    kk, vv = h.kv(0, 0, T)
    o = _decode(h, q, [T], 256, scale)[0]
    x = q[0].double().numpy()
    s = scale * x @ kk.T
    w = np.exp(s - s.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    want = w @ vv
    assert np.abs(want).max() < 2.0 ** (6 - e)  # the large blocks have no part in it
    es = np.log2(np.e) * scale * (np.abs(x) @ np.abs(kk).T).max() * (2.0 ** -22 + 132 * 2.0 ** -24)
    top = np.abs(vv).reshape(-1, 32 * 128).max(axis=1).repeat(32)
    tol = w @ np.abs(vv) * (1.5 * es + 2.0 ** -20 + T * 2.0 ** -24) + T * 2.0 ** -24 * (w * top).max(axis=1, keepdims=True)
    half = {F32: 2.0 ** -24, F16: 2.0 ** -11}[dtype]
    tol += np.abs(want) * half + (2.0 ** -25 if dtype == F16 else 0.0)
    assert (np.abs(o - want) <= tol).all(), (np.abs(o - want) / tol).max()
    assert h.c.status.item() == 0


@pytest.mark.parametrize("live", [1.0, 0.15])
@pytest.mark.parametrize("G,hkv", [(6, 2), (1, 3), (8, 1)])
def test_float32_chunks_of_many_short_sequences(live, G, hkv):
    """More blocks than CTAs, none of them cut, many without a token: every live one is computed, once."""
    r = np.random.default_rng(7)
    batch, n = 60, 19
    cnt = [int(r.integers(1, n + 1)) if r.random() < live else 0 for _ in range(batch)]
    start = [int(r.integers(0, 130)) for _ in range(batch)]
    h = _filled(batch, hkv, 32, 5, "s8", [s + c for s, c in zip(start, cnt)], 80, F32)
    q = torch.randn((batch, n, G * hkv, 128), generator=torch.Generator().manual_seed(4))
    o = _prefill(h, q, start, 160, cnt)
    _check_prefill(h, q, o, start, cnt, F32, stride=4)
    assert h.c.status.item() == 0
    lens = [s if c else 0 for s, c in zip(start, cnt)]  # and decode, sequences of no tokens among them
    o = _decode(h, q[:, 0], lens, 160)
    for b, m in enumerate(lens):
        kv = [h.kv(b, i, m) for i in range(hkv)]
        _check_rows(o[b], q[b, 0].double().numpy(), np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv]), 128 ** -0.5, F32)


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("down", [20.3, 24.6, 26.2, 31.0])
@pytest.mark.parametrize("batch,T", [(1, 700), (40, 700), (1, 3000), (300, 1500)])
def test_keys_far_below_the_first(code, dtype, down, batch, T):
    """Behind a first key with nearly all the weight and V = 0, keys of 2^-down of it that have all of V: decode, and a chunk
    of float32.  Weights times block scales are held in two binary16 terms of steps down to 2^-24, their maximum being 2^14
    or more: a key is off by 2^-39 of that, and a code times scale is at most twice the largest |V|: T 2^-38 in all, beside
    sum w |V| (1.5 e_s + 2^-20 + T 2^-24) and half a step of the output's type."""
    hkv, G = 2, 4
    per = -(-T // 64)
    c = B.PagedCache8(1, hkv, 64, per, code=code, block_table=torch.arange(per, dtype=torch.int32, device=DEV).repeat(batch, 1))
    k, v = torch.zeros((1, T, hkv, 128), device=DEV), torch.ones((1, T, hkv, 128), device=DEV)
    k[:, 0, :, 7] = 240.0
    v[:, 0] = 0.0
    one = B.PagedCache8(1, hkv, 64, per, code=code, block_table=c.block_table[:1].contiguous(), pool=c.pool)
    B.iq_append8(one, 0, k, v, _i32([0]))  # every sequence reads the same pages
    kv = []
    for side in (0, 1):
        x = torch.empty((hkv, T, 128), dtype=F32, device=DEV)
        B.iq_export8(one, 0, side, 0, 0, T, x)
        kv.append(x[0].double().cpu().numpy())
    scale = down * float(np.log(2.0)) / kv[0][0, 7]
    scale = float(np.float32(scale))
    s = scale * kv[0][:, 7]
    w = np.exp(s - s.max())
    w /= w.sum()
    q = torch.zeros((batch, hkv * G, 128), dtype=dtype, device=DEV)
    q[..., 7] = 1.0
    es = np.log2(np.e) * s.max() * (2.0 ** -22 + 132 * 2.0 ** -24)

    def check(o, w, n):
        want = float(w @ kv[1][:n, 0])
        tol = want * (1.5 * es + 2.0 ** -20 + n * 2.0 ** -24) + n * 2.0 ** -38 + want * (2.0 ** -11 if dtype == F16 else 2.0 ** -24)
        tol += 2.0 ** -25 if dtype == F16 else 0.0
        assert np.abs(o - want).max() <= tol, (np.abs(o - want).max() / tol, o.min(), o.max(), want)

    out = torch.full_like(q, float("nan"))
    ws = torch.zeros(B.iq_decode8_workspace_size(batch, hkv * G, hkv, per * 64), dtype=torch.uint8, device=DEV)
    B.iq_decode8_attention(c, 0, q, _i32([T] * batch), per * 64, out, ws, scale)
    check(out.double().cpu().numpy(), w, T)
    if dtype == F32:
        q = q[:, None].repeat(1, 3, 1, 1)
        out = torch.full_like(q, float("nan"))
        ws = torch.zeros(B.iq_prefill8_workspace_size(batch, 3, hkv * G, hkv, per * 64), dtype=torch.uint8, device=DEV)
        B.iq_prefill8_attention(c, 0, q, _i32([T - 3] * batch), per * 64, out, ws, scale=scale)
        for i in range(3):
            n = T - 2 + i
            check(out[:, i].double().cpu().numpy(), w[:n] / w[:n].sum(), n)
    assert c.status.item() == 0


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("apart", [100, 116, 122])
def test_decode_small_weights_of_very_large_values(code, apart):
    """A block whose keys have 2^-apart of the others' weight, and values 2^(apart + 4) times as large: they are what comes
    out."""
    T = 96
    h = Held(1, 1, 96, 1, code, contiguous=True)
    k, v = torch.zeros((1, T, 1, 128)), _tokens(62, (1, T, 1, 128), F32)
    k[:, 32:64, :, 9] = -60.0
    v *= 2.0 ** -64
    v[:, 32:64] *= 2.0 ** (apart + 4)
    q = torch.zeros((1, 4, 128))
    q[..., 9] = 8.0
    h.append(k, v, [0])
    kk, vv = h.kv(0, 0, T)
    scale = float(np.float32(apart * np.log(2.0) / (-kk[32, 9] * 8.0)))
    o = _decode(h, q, [T], 96, scale)[0]
    s = scale * q[0].double().numpy() @ kk.T
    w = np.exp(s - s.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    want, mass = w @ vv, w @ np.abs(vv)
    es = apart * (2.0 ** -22 + 132 * 2.0 ** -24)
    tol = mass * (1.5 * es + 2.0 ** -20 + T * 2.0 ** -24) + T * 2.0 ** -38 * mass.max() * 32 + np.abs(want) * 2.0 ** -24
    assert np.abs(want).max() > 2.0 ** -64 and (np.abs(o - want) <= tol).all(), (np.abs(o - want) / tol).max()
    assert h.c.status.item() == 0
