"""The 8-bit cache on the GPU: appends against the fp64 oracle (values and scales equal to the bit), decode and prefill
attention against fp64 attention over the values that the cache holds, and a run of the calls as a model makes them.

Tolerance of attention, per output value, with V and K the held values, w the softmax weights (they sum to 1) and
u = 2^-24 the half step of float32:
  * scores (log2 units) are off by at most e_s = log2(e) scale sum|q_i k_i| (2^-22 + 132 u): two binary16 terms of q,
    128 products summed in float32, four more roundings; a weight then is off by a factor of 2^(2 e_s) <= 1 + 1.5 e_s;
  * exponentials and the weights' two binary16 terms: 2^-20 together; sums over T tokens: T u;
  * 16-bit outputs of prefill: weights of one binary16 term, 2^-11;
  * rounding of the output: half a step of its type.
All but the last are relative to vmax, the largest |V| of the head."""

import numpy as np
import pytest
import torch

from oracle import cache8
from rotated_bit_kv_iq_b200 import binding as B
from tests._helpers import Guarded, record_parity

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_bit_kv_iq_b200 import build

    build.build()
    B.lib()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tokens(seed, shape, dtype=F16):
    """Channel scales of their own, two outlying channels a head."""
    g = torch.Generator().manual_seed(seed)
    s = torch.exp(0.5 * torch.randn(shape[-2:], generator=g))
    s[:, 5] *= 12
    s[:, 77] *= 12
    return (torch.randn(shape, generator=g) * s).to(dtype)


class Held:
    """A paged cache on the GPU and the oracle's beside it; every pool byte that nothing was written to is 0x7F (NaN codes
    of e4m3) and every scale that was not, NaN."""

    def __init__(self, batch, hkv, ps, per, code, seed=0, contiguous=False):
        self.batch, self.hkv, self.ps, self.per, self.code = batch, hkv, ps, per, code
        g = torch.Generator().manual_seed(seed)
        self.n_pages = batch * per + 3
        self.table = None if contiguous else torch.randperm(self.n_pages, generator=g)[: batch * per].view(
            batch, per).to(torch.int32).to(DEV)
        assert not contiguous or per == 1
        self.pool = Guarded((B.iq_cache8_bytes(2, hkv, ps, self.n_pages),), torch.uint8, fill=0x7F)
        self.c = B.PagedCache8(2, hkv, ps, self.n_pages, block_table=self.table, code=code, pool=self.pool.t)
        self.c.tiles()[..., 8192:8200] = torch.tensor([0, 0, 0xC0, 0x7F] * 2, dtype=torch.uint8, device=DEV)
        self.o = cache8.Cache8(batch, hkv, per * ps, code)

    def append(self, k, v, start, cnt=None, layer=1):
        """k, v on the CPU."""
        B.iq_append8(self.c, layer, None if k is None else k.to(DEV), None if v is None else v.to(DEV), _i32(start),
                     None if cnt is None else _i32(cnt))
        for b in range(self.batch):
            n = (k if k is not None else v).shape[1] if cnt is None else cnt[b]
            for side, x in ((0, k), (1, v)):
                if x is not None:
                    self.o.append(side, b, x[b, :n].double().numpy(), start[b])

    def check(self, lens, layer=1):
        """The first lens[b] tokens are the oracle's, to the bit."""
        for b, n in enumerate(lens):
            for side in (0, 1):
                got = torch.empty((self.hkv, n, 128), dtype=F32, device=DEV)
                B.iq_export8(self.c, layer, side, b, 0, n, got)
                want = np.stack([self.o.values(side, b, h, n) for h in range(self.hkv)]).astype(np.float32)
                np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=f"sequence {b}, side {side}")
        self.pool.check("pool")

    def kv(self, b, h, n):
        return self.o.values(0, b, h, n), self.o.values(1, b, h, n)


def _filled(batch, hkv, ps, per, code, lens, seed, dtype=F16, contiguous=False):
    h = Held(batch, hkv, ps, per, code, seed, contiguous)
    n = max(max(lens), 1)
    k, v = _tokens(seed + 1, (batch, n, hkv, 128), dtype), _tokens(seed + 2, (batch, n, hkv, 128), dtype)
    h.append(k, v, [0] * batch, list(lens))
    return h


def _half_step(dtype):
    return {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}[dtype]


def _check_rows(got, q, k, v, scale, dtype, one_term=False):
    """got, q: [Hq][128] of one query token over k, v [Hkv][T][128]; returns the share of the tolerance used."""
    want = cache8.attention(q, k, v, scale)
    g, T = q.shape[0] // k.shape[0], k.shape[1]
    if T == 0:
        assert not got.any()
        return 0.0
    es = np.log2(np.e) * scale * np.max(np.abs(q)[:, None] @ np.abs(k).repeat(g, 0).transpose(0, 2, 1), axis=(1, 2))
    es = es * (2.0 ** -22 + 132 * 2.0 ** -24)
    vmax = np.abs(v).max(axis=(1, 2)).repeat(g)
    tol = vmax * (1.5 * es + 2.0 ** -20 + T * 2.0 ** -24 + (2.0 ** -11 if one_term else 0.0))
    tol = tol[:, None] + np.abs(want) * _half_step(dtype) + 2.0 ** -24
    bad = np.abs(got - want) / tol
    assert np.isfinite(got).all() and bad.max() <= 1.0, (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    return bad.max()


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("ps,start", [(64, [0, 5, 31, 32]), (96, [63, 0, 33, 95])])
def test_append_is_the_oracles(code, dtype, ps, start):
    h = Held(4, 3, ps, 3, code)
    old = _tokens(1, (4, max(start), 3, 128), dtype)
    h.append(old, old.flip(1), [0] * 4, start)
    for n, cnt in ((1, None), (70, [70, 0, 33, 64])):
        k, v = _tokens(2, (4, n, 3, 128), dtype), 3 * _tokens(3, (4, n, 3, 128), dtype)
        h.append(k, v, start, cnt)
        h.check([s + (n if cnt is None else cnt[b]) for b, s in enumerate(start)])
    assert h.c.status.item() == 0


@pytest.mark.parametrize("code", ["e4m3", "s8"])
def test_append_token_by_token_with_scales_that_grow(code):
    """40 single-token steps whose magnitudes rise, so that blocks grow and are rounded again; one side alone too."""
    h = Held(2, 2, 32, 2, code)
    g = torch.Generator().manual_seed(4)
    for t in range(40):
        x = (torch.randn((2, 1, 2, 128), generator=g) * 1.2 ** t).to(F16)
        h.append(x, None if t % 7 == 3 else -x, [t, t])
        if t % 7 == 3:
            h.append(None, -x, [t, t])
    h.check([40, 40])


def test_append_into_a_block_that_holds_nothing():
    """A start inside a block that was never written: what lies before counts for nothing."""
    h = Held(1, 1, 32, 1, "e4m3", contiguous=True)
    x = _tokens(6, (1, 4, 1, 128))
    B.iq_append8(h.c, 1, x.to(DEV), x.to(DEV), _i32([3]))
    h.o.append(0, 0, x[0].double().numpy(), 0)
    got = torch.empty((1, 7, 128), dtype=F32, device=DEV)
    B.iq_export8(h.c, 1, 0, 0, 0, 7, got)
    assert not got[0, :3].any()
    np.testing.assert_array_equal(got[0, 3:].cpu().numpy(), h.o.values(0, 0, 0, 4).astype(np.float32))


def test_append_extreme_values():
    """Zeros, the largest and smallest numbers, infinities and NaN, which keep to their own coordinates."""
    for dtype, big in ((F16, 65504.0), (BF16, 3e38), (F32, 3e38)):
        for code in ("e4m3", "s8"):
            h = Held(1, 1, 128, 1, code, contiguous=True)
            x = torch.zeros((1, 128, 1, 128))
            x[0, 32:64, 0, :4] = torch.tensor([big, -big, 1.0, 6e-8])
            x[0, 64:96, 0, :5] = torch.tensor([float("inf"), float("-inf"), float("nan"), 2.0, -0.5])
            x[0, 96:, 0] = 6e-8 if dtype == F16 else 1e-37
            x = x.to(dtype)
            h.append(x, x, [0])
            h.check([128])


def test_append_strided_rows_of_a_fused_projection():
    h = Held(3, 2, 64, 2, "e4m3")
    qkv = _tokens(7, (3, 9, 8, 128)).to(DEV)
    k, v = qkv[:, :, 4:6], qkv[:, :, 6:8]
    assert not k.is_contiguous()
    B.iq_append8(h.c, 1, k, v, _i32([0, 40, 100]))
    for b, s in enumerate([0, 40, 100]):
        h.o.append(0, b, k[b].cpu().double().numpy(), s)
        h.o.append(1, b, v[b].cpu().double().numpy(), s)
    for side, x in ((0, k), (1, v)):
        got = torch.empty((2, 9, 128), dtype=F32, device=DEV)
        B.iq_export8(h.c, 1, side, 0, 0, 9, got)
        np.testing.assert_array_equal(got.cpu().numpy(), np.stack([h.o.values(side, 0, i, 9) for i in range(2)]).astype(np.float32))


def test_append_bad_positions_and_pages_are_skipped_and_flagged():
    h = Held(4, 1, 32, 2, "s8")
    h.table[2, 1] = h.n_pages  # outside the pool
    x = _tokens(8, (4, 40, 1, 128))
    before = h.pool.t.clone()
    B.iq_append8(h.c, 1, x.to(DEV), x.to(DEV), _i32([-8, 30, 0, 64]), _i32([40, 40, 40, 1]))
    torch.cuda.synchronize()
    assert h.c.status.item() == B.IQ_DEVERR_POSITION | B.IQ_DEVERR_PAGE
    h.pool.check("pool")
    changed = (h.pool.t != before).view(2, h.n_pages, -1).any(-1).cpu()
    t = h.table.cpu()
    want = {int(t[0, 0]), int(t[1, 0]), int(t[1, 1]), int(t[2, 0])}
    assert set(changed[1].nonzero().flatten().tolist()) == want and not changed[0].any()
    h.o.append(0, 0, x[0, 8:].double().numpy(), 0)  # the eight before position 0 are left out
    got = torch.empty((1, 32, 128), dtype=F32, device=DEV)
    B.iq_export8(h.c, 1, 0, 0, 0, 32, got)
    np.testing.assert_array_equal(got[0].cpu().numpy(), h.o.values(0, 0, 0, 32).astype(np.float32))
    h.c.status.zero_()
    B.iq_append8(h.c, 1, x.to(DEV), None, _i32([0, 0, 0, 0]), _i32([41, -1, 0, 0]))
    assert h.c.status.item() == B.IQ_DEVERR_CTX


# ---------------------------------------------------------------------------------------------- decode
def _decode(h, q, lens, max_ctx, scale=None, layer=1):
    out = Guarded(q.shape, q.dtype, fill=float("nan"))
    ws = Guarded((B.iq_decode8_workspace_size(q.shape[0], q.shape[1], h.hkv, max_ctx),), torch.uint8, fill=0)
    for _ in range(2):  # the workspace is left ready
        B.iq_decode8_attention(h.c, layer, q.to(DEV), _i32(lens), max_ctx, out.t, ws.t, scale)
        torch.cuda.synchronize()
        if _ == 0:
            first = out.t.clone()
    assert torch.equal(first.view(torch.uint8), out.t.view(torch.uint8)), "the same call, another result"
    out.check("out")
    ws.check("workspace")
    return out.t.double().cpu().numpy()


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_decode_matches_fp64(code, dtype, G):
    """No token, one, a tile less one, a tile, one more, and a long one over ragged pages, in one batch."""
    lens = [0, 1, 31, 32, 33, 421]
    h = _filled(6, 2, 96, 5, code, lens, 10 + G, dtype)
    q = torch.randn((6, 2 * G, 128), generator=torch.Generator().manual_seed(G)).to(dtype)
    o = _decode(h, q, lens, 480)
    used = 0.0
    for b, n in enumerate(lens):
        kv = [h.kv(b, i, n) for i in range(2)]
        used = max(used, _check_rows(o[b], q[b].double().numpy(), np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv]),
                                     128 ** -0.5, dtype))
    assert h.c.status.item() == 0
    print(f"decode8 {code} {dtype} G={G}: {100 * used:.0f}% of the tolerance")


@pytest.mark.parametrize("batch,hkv,lens", [(1, 1, [4000]), (1, 4, [2500]), (40, 2, None), (300, 1, None)])
def test_decode_over_many_splits_and_many_sequences(batch, hkv, lens):
    """A context split over many CTAs; more sequences than a CTA scans at once, most of them short."""
    g = np.random.default_rng(5)
    lens = lens or [int(x) for x in g.integers(0, 70, batch)]
    per = -(-max(lens) // 64)
    h = _filled(batch, hkv, 64, per, "e4m3", lens, 30)
    q = torch.randn((batch, 4 * hkv, 128), generator=torch.Generator().manual_seed(1)).to(F32)
    o = _decode(h, q, lens, per * 64, 0.05)
    for b, n in enumerate(lens):
        kv = [h.kv(b, i, n) for i in range(hkv)]
        _check_rows(o[b], q[b].double().numpy(), np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv]), 0.05, F32)


@pytest.mark.parametrize("code", ["e4m3", "s8"])
def test_decode_with_many_tiles_a_cta(code):
    """More tiles to a CTA than it has in flight at once, in segments of several groups, some of a tile or two."""
    lens = [6000, 33, 5000, 1, 7001, 0, 6400, 64, 4097]
    hkv, ps, per = 4, 64, 112
    c = B.PagedCache8(1, hkv, ps, len(lens) * per, code=code, block_table=torch.randperm(
        len(lens) * per, generator=torch.Generator().manual_seed(3)).view(-1, per).to(torch.int32).to(DEV))
    c.pool.fill_(0x7F)
    k, v = (_tokens(s, (len(lens), max(lens), hkv, 128)).to(DEV) for s in (4, 5))
    B.iq_append8(c, 0, k, v, _i32([0] * len(lens)), _i32(lens))
    for G, dtype in ((4, F16), (8, F32)):
        q = torch.randn((len(lens), G * hkv, 128), generator=torch.Generator().manual_seed(2)).to(dtype)
        out = torch.full_like(q, float("nan")).to(DEV)
        ws = torch.zeros(B.iq_decode8_workspace_size(len(lens), G * hkv, hkv, ps * per), dtype=torch.uint8, device=DEV)
        for _ in range(3):
            B.iq_decode8_attention(c, 0, q.to(DEV), _i32(lens), ps * per, out, ws)
        o = out.double().cpu().numpy()
        assert c.status.item() == 0
        for b, n in enumerate(lens):
            kv = []
            for side in (0, 1):
                x = torch.empty((hkv, n, 128), dtype=F32, device=DEV)
                B.iq_export8(c, 0, side, b, 0, n, x)
                kv.append(x.double().cpu().numpy())
            _check_rows(o[b], q[b].double().numpy(), *kv, 128 ** -0.5, dtype)


def test_decode_calls_of_several_sizes_share_a_workspace():
    """One workspace, large enough for each: a long sequence of one head, cut over all CTAs, then many groups."""
    n, batch, hkv, ps, per = 20000, 40, 8, 64, 16
    one = B.PagedCache8(1, 1, 64, 320, block_table=torch.arange(320, dtype=torch.int32, device=DEV).view(1, -1))
    many = B.PagedCache8(1, hkv, ps, batch * per,
                         block_table=torch.arange(batch * per, dtype=torch.int32, device=DEV).view(batch, per))
    B.iq_append8(one, 0, *(_tokens(s, (1, n, 1, 128)).to(DEV) for s in (50, 51)), _i32([0]))
    B.iq_append8(many, 0, *(_tokens(s, (batch, ps * per, hkv, 128)).to(DEV) for s in (52, 53)), _i32([0] * batch))
    q1 = torch.randn((1, 8, 128), generator=torch.Generator().manual_seed(2)).to(F16).to(DEV)
    q2 = torch.randn((batch, 4 * hkv, 128), generator=torch.Generator().manual_seed(3)).to(F16).to(DEV)
    l1, l2 = _i32([n]), _i32([ps * per - 7 * i for i in range(batch)])
    size = max(B.iq_decode8_workspace_size(1, 8, 1, 20480), B.iq_decode8_workspace_size(batch, 4 * hkv, hkv, ps * per))
    shared = torch.zeros(size, dtype=torch.uint8, device=DEV)

    def run(ws):
        a, b = torch.full_like(q1, float("nan")), torch.full_like(q2, float("nan"))
        B.iq_decode8_attention(one, 0, q1, l1, 20480, a, ws)
        B.iq_decode8_attention(many, 0, q2, l2, ps * per, b, ws if ws is shared else torch.zeros_like(ws))
        return a, b

    a, b = run(torch.zeros_like(shared))
    for _ in range(3):
        x, y = run(shared)
        assert torch.equal(x, a) and torch.equal(y, b)
    assert one.status.item() == 0 and many.status.item() == 0
    assert not torch.isnan(a).any() and not torch.isnan(b).any()


@pytest.mark.parametrize("lens", [[0, 0], [1, 0], [40, 700], [3, 260]])
def test_lengths_far_below_the_bound(lens):
    """max_ctx sizes the grid; the lengths decide what there is to share out."""
    h = _filled(2, 1, 64, 200, "e4m3", lens, 42)
    q = torch.randn((2, 4, 128), generator=torch.Generator().manual_seed(2)).to(F16)
    o = _decode(h, q, lens, 12800)
    for b, n in enumerate(lens):
        k, v = h.kv(b, 0, n)
        _check_rows(o[b], q[b].double().numpy(), k[None], v[None], 128 ** -0.5, F16)
    assert h.c.status.item() == 0
    for dtype in (F16, F32):
        q = torch.randn((2, 3, 4, 128), generator=torch.Generator().manual_seed(2)).to(dtype)
        start, cnt = [max(0, n - 3) for n in lens], [min(3, n) for n in lens]
        o = _prefill(h, q, start, 12800, cnt)
        _check_prefill(h, q, o, start, cnt, dtype)
    assert h.c.status.item() == 0


def test_decode_contiguous_cache_and_lengths_out_of_range():
    h = _filled(3, 2, 128, 1, "s8", [128, 60, 5], 40, contiguous=True)
    q = torch.randn((3, 2, 128), generator=torch.Generator().manual_seed(2)).to(BF16)
    o = _decode(h, q, [1000, 60, -4], 128)  # clamped to 128 and 0
    assert h.c.status.item() == B.IQ_DEVERR_CTX
    for b, n in enumerate([128, 60, 0]):
        kv = [h.kv(b, i, n) for i in range(2)]
        _check_rows(o[b], q[b].double().numpy(), np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv]), 128 ** -0.5, BF16)


def test_decode_pages_outside_the_pool_are_left_out():
    h = _filled(2, 1, 32, 3, "e4m3", [96, 70], 41)
    h.table[0, 1] = -1
    h.table[1] = h.n_pages + 7
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(2)).to(F32)
    o = _decode(h, q, [96, 70], 96)
    assert h.c.status.item() == B.IQ_DEVERR_PAGE and not o[1].any()
    k, v = h.kv(0, 0, 96)
    keep = np.r_[0:32, 64:96]
    _check_rows(o[0], q[0].double().numpy(), k[None, keep], v[None, keep], 128 ** -0.5, F32)


def test_decode_scales_far_apart():
    """Blocks whose V (or K) scales differ by 2^20 and more: neither end loses anything."""
    for code in ("e4m3", "s8"):
        h = Held(1, 1, 256, 1, code, contiguous=True)
        k, v = _tokens(50, (1, 256, 1, 128), F32), _tokens(51, (1, 256, 1, 128), F32)
        v[:, :64] *= 2.0 ** 30
        v[:, 64:128] *= 2.0 ** -30
        k[:, 128:] *= 2.0 ** -12
        q = torch.randn((1, 3, 128), generator=torch.Generator().manual_seed(3))
        h.append(k, v, [0])
        kk, vv = h.kv(0, 0, 256)
        o = _decode(h, q, [256], 256)
        _check_rows(o[0], q[0].double().numpy(), kk[None], vv[None], 128 ** -0.5, F32)
        # where the small values have all the weight, they come out whole: the small block's keys and nothing else
        o = _decode(h, q, [64], 256)
        _check_rows(o[0], q[0].double().numpy(), kk[None, :64], vv[None, :64], 128 ** -0.5, F32)


# --------------------------------------------------------------------------------------------- prefill
def _prefill(h, q, start, max_ctx, cnt=None, scale=None, fill=7.0):
    out = Guarded(q.shape, q.dtype, fill=fill)
    ws = Guarded((B.iq_prefill8_workspace_size(q.shape[0], q.shape[1], q.shape[2], h.hkv, max_ctx),), torch.uint8, fill=0x5B)
    for _ in range(2):
        B.iq_prefill8_attention(h.c, 1, q.to(DEV), _i32(start), max_ctx, out.t, ws.t, None if cnt is None else _i32(cnt), scale)
        torch.cuda.synchronize()
        if _ == 0:
            first = out.t.clone()
    assert torch.equal(first.view(torch.uint8), out.t.view(torch.uint8)), "the same call, another result"
    out.check("out")
    ws.check("workspace")
    return out.t.double().cpu().numpy()


def _check_prefill(h, q, o, start, cnt, dtype, scale=128 ** -0.5, fill=7.0, stride=1):
    used = 0.0
    for b, s in enumerate(start):
        assert (o[b, cnt[b]:] == fill).all()
        for i in range(0, cnt[b], stride):
            kv = [h.kv(b, x, s + i + 1) for x in range(h.hkv)]
            used = max(used, _check_rows(o[b, i], q[b, i].double().numpy(), np.stack([x[0] for x in kv]),
                                         np.stack([x[1] for x in kv]), scale, dtype, one_term=dtype != F32))
    return used


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("G", [1, 3, 4, 6, 8])
def test_prefill_matches_fp64(code, dtype, G):
    """Chunks of 37, 1, no and 20 tokens at odd positions of ragged pages; rows behind them stay as they were."""
    start, cnt = [0, 95, 17, 200], [37, 1, 0, 20]
    h = _filled(4, 2, 96, 3, code, [s + c for s, c in zip(start, cnt)], 60 + G, dtype)
    q = torch.randn((4, 37, 2 * G, 128), generator=torch.Generator().manual_seed(G)).to(dtype)
    o = _prefill(h, q, start, 240, cnt)
    used = _check_prefill(h, q, o, start, cnt, dtype)
    assert h.c.status.item() == 0
    print(f"prefill8 {code} {dtype} G={G}: {100 * used:.0f}% of the tolerance")


@pytest.mark.parametrize("dtype,code", [(F16, "e4m3"), (BF16, "s8"), (F32, "e4m3")])
@pytest.mark.parametrize("n,start", [(1, 0), (1, 640), (2, 31), (130, 0), (129, 511), (64, 64)])
def test_prefill_lengths(n, start, dtype, code):
    """One token, chunks around the sizes of tiles and steps, from the start and far in."""
    h = _filled(1, 2, 64, 11, code, [start + n], 80, dtype)
    q = torch.randn((1, n, 8, 128), generator=torch.Generator().manual_seed(n)).to(dtype)
    o = _prefill(h, q, [start], 704)
    _check_prefill(h, q, o, [start], [n], dtype, stride=max(1, n // 40))


def test_prefill_long_chunk_of_a_whole_prompt():
    h = _filled(1, 1, 64, 16, "e4m3", [1000], 81, BF16)
    q = torch.randn((1, 1000, 4, 128), generator=torch.Generator().manual_seed(9)).to(BF16)
    o = _prefill(h, q, [0], 1024, scale=0.07)
    _check_prefill(h, q, o, [0], [1000], BF16, scale=0.07, stride=61)


def test_prefill_out_of_range_starts_and_counts_are_clamped():
    h = _filled(3, 1, 64, 2, "s8", [128, 128, 128], 82)
    q = torch.randn((3, 5, 4, 128), generator=torch.Generator().manual_seed(9)).to(F16)
    o = _prefill(h, q, [-3, 500, 40], 128, [5, 5, 9])
    assert h.c.status.item() == B.IQ_DEVERR_CTX
    _check_prefill(h, q, o, [0, 123, 40], [5, 5, 5], F16)


def test_prefill_pages_outside_the_pool_are_left_out():
    h = _filled(2, 1, 32, 4, "e4m3", [100, 100], 83)
    h.table[0, 1] = -1
    h.table[1] = 10 ** 6
    q = torch.randn((2, 4, 8, 128), generator=torch.Generator().manual_seed(2)).to(F32)
    o = _prefill(h, q, [96, 96], 128)
    assert h.c.status.item() == B.IQ_DEVERR_PAGE and not o[1].any()
    for i in range(4):
        k, v = h.kv(0, 0, 97 + i)
        keep = np.r_[0:32, 64:97 + i]
        _check_rows(o[0, i], q[0, i].double().numpy(), k[None, keep], v[None, keep], 128 ** -0.5, F32)


def test_prefill_scales_far_apart():
    for dtype in (F32, BF16):
        h = Held(1, 1, 256, 1, "e4m3", contiguous=True)
        k, v = _tokens(90, (1, 256, 1, 128), F32), _tokens(91, (1, 256, 1, 128), F32)
        v[:, 32:64] *= 2.0 ** 30
        v[:, 96:160] *= 2.0 ** -20
        k[:, 128:] *= 2.0 ** -12
        h.append(k, v, [0])
        q = torch.randn((1, 250, 2, 128), generator=torch.Generator().manual_seed(3)).to(dtype)
        o = _prefill(h, q, [0], 256)
        _check_prefill(h, q, o, [0], [250], dtype, stride=7)


@pytest.mark.parametrize("code", ["e4m3", "s8"])
def test_prefill_scales_at_the_ends_of_their_range(code):
    """V scales 2^96 apart, or blocks of zeros, are within what 16-bit queries take; farther ones are flagged.  Decode
    takes any."""
    for up, down, flag in ((48, 48, 0), (0, None, 0), (70, 70, B.IQ_DEVERR_RANGE)):
        h = Held(1, 1, 256, 1, code, contiguous=True)
        k, v = _tokens(92, (1, 256, 1, 128), F32), _tokens(93, (1, 256, 1, 128), F32)
        v[:, 32:64] *= 2.0 ** up
        v[:, 96:160] *= 0.0 if down is None else 2.0 ** -down
        if down is None:
            v[:, :32] = 0.0
        k[:, 32:64] *= 8.0  # scores far above and far below the others'
        h.append(k, v, [0])
        q = torch.randn((1, 250, 2, 128), generator=torch.Generator().manual_seed(4)).to(BF16)
        o = _prefill(h, q, [0], 256)
        if not flag:
            _check_prefill(h, q, o, [0], [250], BF16, stride=7)
        assert h.c.status.item() == flag
        h.c.status.zero_()
        kk, vv = h.kv(0, 0, 256)
        _check_rows(_decode(h, q[:, 0].to(F32), [256], 256)[0], q[0, 0].double().numpy(), kk[None], vv[None], 128 ** -0.5, F32)
        assert h.c.status.item() == 0


# ------------------------------------------------------------------------------- streams, graphs, one run
def test_calls_on_another_stream_and_in_graphs():
    """append -> decode captured into two graphs that share a workspace, replayed in turn on a side stream."""
    h = _filled(2, 2, 64, 4, "e4m3", [40, 90], 100)
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(4)).to(F16).to(DEV)
    new = _tokens(101, (2, 1, 2, 128)).to(DEV)
    pos, lens = _i32([40, 90]), _i32([41, 91])
    outs = [torch.zeros_like(q) for _ in range(2)]
    ws = torch.zeros(B.iq_decode8_workspace_size(2, 8, 2, 256), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            B.iq_append8(h.c, 1, new, new, pos)
            B.iq_decode8_attention(h.c, 1, q, lens, 256, outs[i], ws)
            pos.add_(1)
            lens.add_(1)
        graphs.append(g)
    with torch.cuda.stream(side):
        for i in range(6):
            graphs[i % 2].replay()
    side.synchronize()
    assert pos.tolist() == [46, 96] and h.c.status.item() == 0
    for i in range(6):
        for b in range(2):
            x = new[b].cpu().double().numpy()
            h.o.append(0, b, x, [40, 90][b] + i)
            h.o.append(1, b, x, [40, 90][b] + i)
        if i < 4:
            continue
        for b in range(2):
            n = [41, 91][b] + i
            kv = [h.kv(b, j, n) for j in range(2)]
            _check_rows(outs[i % 2][b].double().cpu().numpy(), q[b].double().cpu().numpy(), np.stack([x[0] for x in kv]),
                        np.stack([x[1] for x in kv]), 128 ** -0.5, F16)
    # an explicit stream, also as a number
    o2 = torch.zeros_like(q)
    B.iq_decode8_attention(h.c, 1, q, _i32([46, 96]), 256, o2, ws, stream=side)
    side.synchronize()
    assert torch.equal(o2, outs[1])


def test_a_prompt_and_steps_with_forked_sequences():
    """As a model serves: a prompt is rotated, appended and attended; the sequence is forked; both go on by steps of
    their own; the pool is compacted between.  Checked against fp64 over what the caches should hold."""
    from oracle import rope

    hq, hkv, ps, P = 8, 2, 64, 12
    pt = B.PageTable(4, 4, ps, P)
    cache = B.PagedCache8(1, hkv, ps, P, block_table=pt.block_table, code="e4m3")
    cache.pool.fill_(0x7F)
    pools = B.PagePool.of(cache)
    freq_np, ms = B.iq_rope_frequencies(128, 10000.0, "yarn", 4.0, 64.0, 1.0, 8.0)
    freq = torch.from_numpy(freq_np).to(DEV)
    n0 = 90
    B.iq_pages_extend(pt, _i32([3]), _i32([40]))  # a sequence that leaves holes
    B.iq_pages_extend(pt, _i32([1]), _i32([n0]))
    g = torch.Generator().manual_seed(7)

    def make(n):
        return torch.randn((n, hq + 2 * hkv, 128), generator=g).to(F16).to(DEV)

    held = {}  # sequence -> (k, v) as appended, and the oracle's block-by-block cache

    def turn(qkv, pos):
        q, k = torch.empty_like(qkv[:, :hq]), torch.empty_like(qkv[:, hq:hq + hkv])
        B.iq_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], _i32(pos), freq, q, k, mscale=ms)
        want = rope.rotate(qkv[:, hq:hq + hkv].cpu().double().numpy(), pos, freq_np, "half", ms)
        assert np.abs(k.double().cpu().numpy() - want).max() <= 2.0 ** -11 * np.abs(want).max() + 1e-5
        return q, k, qkv[:, hq + hkv:]

    # the prompt, as sequence 1 of a batch whose other rows are empty
    qkv = make(n0)
    q, k, v = turn(qkv, list(range(n0)))
    K, V, Q = (torch.zeros((4, n0) + x.shape[1:], dtype=F16, device=DEV) for x in (k, v, q))
    K[1], V[1], Q[1] = k, v, q
    cnt = _i32([0, n0, 0, 0])
    B.iq_append8(cache, 0, K, V, _i32([0, 0, 0, 0]), cnt)
    o = torch.zeros_like(Q)
    ws = torch.zeros(B.iq_prefill8_workspace_size(4, n0, hq, hkv, 256), dtype=torch.uint8, device=DEV)
    B.iq_prefill8_attention(cache, 0, Q, _i32([0, 0, 0, 0]), 256, o, ws, cnt)
    ref = cache8.Cache8(4, hkv, 256, "e4m3")
    ref.append(0, 1, k.cpu().double().numpy(), 0)
    ref.append(1, 1, v.cpu().double().numpy(), 0)
    for i in (0, 31, 32, 89):
        kv = [(ref.values(0, 1, x, i + 1), ref.values(1, 1, x, i + 1)) for x in range(hkv)]
        _check_rows(o[1, i].double().cpu().numpy(), q[i].double().cpu().numpy(), np.stack([x[0] for x in kv]),
                    np.stack([x[1] for x in kv]), 128 ** -0.5, F16, one_term=True)
    # fork into 0 and 2, let 3 go, close the holes
    B.iq_pages_fork(pt, pools, _i32([1, 1]), _i32([0, 2]))
    for s in (0, 2):
        ref.codes[:, s], ref.scales[:, s] = ref.codes[:, 1], ref.scales[:, 1]
    B.iq_pages_free(pt, _i32([3]))
    n_held = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.iq_pages_compact(pt, pools, n_held)
    assert n_held.item() == 4 and pt.block_table.max().item() == 3 and pt.status.item() == 0  # 1 full page and 3 tails
    # six steps of 0, 1 and 2 with tokens of their own
    wsd = torch.zeros(B.iq_decode8_workspace_size(4, hq, hkv, 256), dtype=torch.uint8, device=DEV)
    for t in range(n0, n0 + 45):
        B.iq_pages_extend(pt, _i32([0, 1, 2]), _i32([t + 1] * 3))
        q, k, v = turn(make(4), [t] * 4)
        one = _i32([1, 1, 1, 0])
        B.iq_append8(cache, 0, k[:, None], v[:, None], _i32([t] * 4), one)
        out = torch.empty_like(q)
        B.iq_decode8_attention(cache, 0, q, pt.seq_len, 256, out, wsd)
        for s in range(3):
            ref.append(0, s, k[s:s + 1].cpu().double().numpy(), t)
            ref.append(1, s, v[s:s + 1].cpu().double().numpy(), t)
            if t % 11 == 0 or t == n0 + 44:
                kv = [(ref.values(0, s, x, t + 1), ref.values(1, s, x, t + 1)) for x in range(hkv)]
                _check_rows(out[s].double().cpu().numpy(), q[s].double().cpu().numpy(), np.stack([x[0] for x in kv]),
                            np.stack([x[1] for x in kv]), 128 ** -0.5, F16)
        assert not out[3].any()
    assert cache.status.item() == 0 and pt.status.item() == 0
    record_parity("8-bit cache: prompt, fork, compaction and 45 steps (own tolerance)")
