"""Prefill of 16-bit queries over the 8-bit cache where a CTA has many steps of 128 keys, several blocks, and scores whose
maximum moves: against attention in fp64 over the values that the cache holds, read back by iq_export8.

Tolerance of a value, with w the softmax weights, V the held values, u = 2^-24 and T keys:
  * scores (log2 units) are off by at most e_s = log2(e) scale sum|q_i k_i| (2^-22 + 132 u), the weights by a factor of
    1 + 1.5 e_s; exponentials and their arguments 2^-20; float32 sums over T keys T u; a weight as one binary16 number
    2^-11, all of these relative to sum w |V|;
  * a weight below binary16's normal numbers is off by half their step, 2^-25, of units of 2^-8 of the largest weight times V
    scale that the row has met; a scale times the largest code is at most twice the largest |V| of its block: T 2^-32 vtop,
    vtop the largest |V| held;
  * rounding of the output: half a step of its type."""

import numpy as np
import pytest
import torch

from rotated_bit_kv_iq_b200 import binding as B
from tests._helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF_STEP = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_bit_kv_iq_b200 import build

    build.build()
    B.lib()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tokens(seed, shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device=DEV))
    s[:, 5] *= 12
    s[:, 77] *= 12
    return torch.randn(shape, generator=g, device=DEV) * s


class Cache:
    """One layer of a paged cache on shuffled pages; what nothing was written to is 0x7F (NaN codes of e4m3), its scales NaN."""

    def __init__(self, batch, hkv, ps, per, code, seed=0):
        n_pages = batch * per + 2
        self.hkv, self.per, self.ps, self.n_pages = hkv, per, ps, n_pages
        self.table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))[: batch * per].view(
            batch, per).to(torch.int32).to(DEV)
        self.c = B.PagedCache8(1, hkv, ps, n_pages, block_table=self.table, code=code)
        self.c.pool.fill_(0x7F)
        self.c.tiles()[..., 8192:8200] = torch.tensor([0, 0, 0xC0, 0x7F] * 2, dtype=torch.uint8, device=DEV)

    def append(self, k, v, cnt=None):
        B.iq_append8(self.c, 0, k, v, _i32([0] * k.shape[0]), None if cnt is None else _i32(cnt))

    def held(self, b, n):
        """K, V of the first n tokens of sequence b, float64 [Hkv][n][128]."""
        kv = [torch.empty((self.hkv, n, 128), device=DEV) for _ in range(2)]
        for side in (0, 1):
            B.iq_export8(self.c, 0, side, b, 0, n, kv[side])
        return [x.double() for x in kv]


def _prefill(cache, q, start, max_ctx, cnt=None, scale=None, fill=7.0):
    out = Guarded(q.shape, q.dtype, fill=fill)
    ws = Guarded((B.iq_prefill8_workspace_size(*q.shape[:3], cache.hkv, max_ctx),), torch.uint8, fill=0x5B)
    first = None
    for _ in range(2):
        B.iq_prefill8_attention(cache.c, 0, q, _i32(start), max_ctx, out.t, ws.t, None if cnt is None else _i32(cnt), scale)
        torch.cuda.synchronize()
        if first is None:
            first = out.t.clone()
    assert torch.equal(first.view(torch.uint8), out.t.view(torch.uint8)), "the same call, another result"
    out.check("out")
    ws.check("workspace")
    return out.t


def _check(cache, q, o, start, cnt, scale=128 ** -0.5, rows=48, gone=None, fill=7.0):
    """Some rows of every sequence; gone: {sequence: bool mask of the keys that are not there}.  The largest share of the
    tolerance that is used."""
    used = 0.0
    for b, (s, n) in enumerate(zip(start, cnt)):
        assert (o[b, n:] == fill).all()
        if n == 0:
            continue
        T = s + n
        k, v = cache.held(b, T)
        g = q.shape[2] // cache.hkv
        there = torch.ones(T, dtype=torch.bool, device=DEV)
        if gone and b in gone:
            there &= ~gone[b][:T].to(DEV)
            k[:, ~there], v[:, ~there] = 0.0, 0.0
        k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
        vtop = v.abs().amax((1, 2))[:, None]
        at = sorted({0, n - 1, *np.linspace(0, n - 1, rows).astype(int).tolist()})
        for i in at:
            x = q[b, i].double()
            sc = scale * torch.einsum("htd,hd->ht", k, x)
            see = there & (torch.arange(T, device=DEV) <= s + i)
            got = o[b, i].double()
            if not see.any():
                assert not got.any(), (b, i)
                continue
            w = torch.softmax(sc.masked_fill(~see, float("-inf")), dim=1)
            want, mass = torch.einsum("ht,htd->hd", w, v), torch.einsum("ht,htd->hd", w, v.abs())
            es = np.log2(np.e) * scale * torch.einsum("htd,hd->ht", k.abs(), x.abs()).masked_fill(~see, 0.0).amax(1)[:, None]
            es = es * (2.0 ** -22 + 132 * 2.0 ** -24)
            tol = mass * (1.5 * es + 2.0 ** -20 + T * 2.0 ** -24 + 2.0 ** -11) + T * 2.0 ** -32 * vtop
            tol = tol + want.abs() * HALF_STEP[q.dtype] + (2.0 ** -25 if q.dtype == F16 else 0.0)
            assert torch.isfinite(got).all(), (b, i)
            share = ((got - want).abs() / tol.clamp_min(1e-300)).max().item()  # (values of zeros: neither may be off)
            assert share <= 1.0, (b, i, share)
            used = max(used, share)
    return used


def _q(seed, shape, dtype):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


@pytest.mark.parametrize("dtype,code", [(F16, "e4m3"), (BF16, "s8")])
@pytest.mark.parametrize("G,n", [(4, 3000), (7, 2100), (1, 3100)])
def test_a_long_prompt_of_two_heads(dtype, code, G, n):
    """More steps than SMs: a CTA reuses its K, V and score buffers and takes several blocks, whole and cut."""
    c = Cache(1, 2, 64, -(-n // 64), code)
    k, v = _tokens(1, (1, n, 2, 128)).to(dtype), _tokens(2, (1, n, 2, 128)).to(dtype)
    c.append(k, v)
    q = _q(3, (1, n, 2 * G, 128), dtype)
    o = _prefill(c, q, [0], c.per * 64)
    used = _check(c, q, o, [0], [n], rows=64)
    assert c.c.status.item() == 0
    print(f"{100 * used:.0f}% of the tolerance")


@pytest.mark.parametrize("dtype,code", [(BF16, "e4m3"), (F16, "s8")])
def test_a_ragged_batch_with_long_contexts(dtype, code):
    """Sequences of very different lengths and counts, none and one among them, on pages of 96 tokens."""
    start, cnt, n, hkv = [0, 2500, 7, 5000, 130, 6001], [1500, 701, 0, 1, 33, 1499], 1500, 2
    lens = [s + c for s, c in zip(start, cnt)]
    c = Cache(6, hkv, 96, -(-max(lens) // 96), code, seed=1)
    k, v = _tokens(4, (6, max(lens), hkv, 128)).to(dtype), _tokens(5, (6, max(lens), hkv, 128)).to(dtype)
    c.append(k, v, lens)
    q = _q(6, (6, n, 6, 128), dtype)
    o = _prefill(c, q, start, c.per * 96, cnt)
    _check(c, q, o, start, cnt, rows=24)
    assert c.c.status.item() == 0


@pytest.mark.parametrize("dtype,code", [(F16, "e4m3"), (BF16, "s8")])
@pytest.mark.parametrize("jumps", [[1500, 2600], [70, 1111, 2047, 2911], [64, 96, 2943, 2944, 2990], [2999]])
def test_scores_that_rise_late_in_the_context(dtype, code, jumps):
    """At each of these positions the keys' scores rise by 24 log2 units for good: what was summed before is scaled down,
    and what a row's last half-step brings has nearly all the weight."""
    n, hkv, scale = 3000, 2, 0.11
    c = Cache(1, hkv, 64, -(-n // 64), code)
    k, v = 0.3 * _q(7, (1, n, hkv, 128), F32), _tokens(8, (1, n, hkv, 128))
    k[..., 3] = 0.0
    for j in jumps:
        k[:, j:, :, 3] += 24.0 / (np.log2(np.e) * scale * 8.0)
    c.append(k.to(dtype), v.to(dtype))
    q = _q(9, (1, n, 4 * hkv, 128), dtype)
    q[..., 3] = 8.0
    q[:, :, 1::4, 3] = -8.0  # and a head whose scores fall
    o = _prefill(c, q, [0], c.per * 64, scale=scale)
    _check(c, q, o, [0], [n], scale=scale, rows=96)
    assert c.c.status.item() == 0


@pytest.mark.parametrize("dtype,code", [(F16, "s8"), (BF16, "e4m3")])
def test_scores_that_rise_with_values_that_fall(dtype, code):
    """V scales that change by 2^5 or 2^12 and more from block to block under scores that change too: neither order loses the
    row's maximum."""
    n, hkv = 1400, 2
    c = Cache(1, hkv, 32, -(-n // 32), code)
    k, v = _tokens(10, (1, n, hkv, 128)), _tokens(11, (1, n, hkv, 128))
    step = torch.arange(n, device=DEV) // 32
    v *= torch.exp2((5.0 if dtype == F16 else 12.0) * ((step * 7) % 5 - 2).float())[None, :, None, None]
    k *= torch.exp2(((step * 3) % 4 - 2).float())[None, :, None, None]
    v = v.clamp(-6e4, 6e4) if dtype == F16 else v
    c.append(k.to(dtype), v.to(dtype))
    q = _q(12, (1, n, 4 * hkv, 128), dtype)
    o = _prefill(c, q, [0], c.per * 32, scale=0.05)
    _check(c, q, o, [0], [n], scale=0.05, rows=96)
    assert c.c.status.item() == 0


@pytest.mark.parametrize("dtype,code", [(F16, "e4m3"), (BF16, "s8"), (BF16, "e4m3"), (F16, "s8")])
def test_pages_outside_the_pool_with_16_bit_queries(dtype, code):
    """Sequences without their first pages, without pages in the middle (more than a CTA's share of the steps), without
    any, and with one page only."""
    start, cnt = [3500, 3950, 100, 0], [130, 33, 60, 90]
    lens = [s + c for s, c in zip(start, cnt)]
    c = Cache(4, 1, 32, 128, code, seed=2)
    c.append(_tokens(13, (4, max(lens), 1, 128)).to(dtype), _tokens(14, (4, max(lens), 1, 128)).to(dtype), lens)
    q = _q(15, (4, max(cnt), 8, 128), dtype)
    good = _prefill(c, q, start, 4096, cnt)  # with all pages
    _check(c, q, good, start, cnt, rows=16)
    assert c.c.status.item() == 0
    gone = {b: torch.zeros(4096, dtype=torch.bool) for b in range(4)}

    def drop(b, p0, p1, page):
        gone[b][32 * p0: 32 * p1] = True
        return c.table[b, p0:p1].clone(), b, p0, p1, page

    lost = [drop(0, 0, 5, -1), drop(0, 30, 111, c.n_pages), drop(1, 0, 123, 10 ** 9), drop(2, 0, 5, -7), drop(3, 0, 2, -1)]
    keep = c.table.clone()
    for _, b, p0, p1, page in lost:
        c.table[b, p0:p1] = page
    o = _prefill(c, q, start, 4096, cnt)
    assert c.c.status.item() == B.IQ_DEVERR_PAGE
    assert not o[2, : cnt[2]].any()
    c.table.copy_(keep)
    _check(c, q, o, start, cnt, rows=40, gone=gone)


@pytest.mark.parametrize("down", [24.6, 25.2, 29.0])
@pytest.mark.parametrize("dtype,code", [(F16, "e4m3"), (BF16, "s8")])
def test_many_keys_far_below_the_first(dtype, code, down):
    """Behind a first key with nearly all the weight and V = 0, thousands of keys of 2^-24.6 of it and less that have all of
    V: blocks enough that a CTA goes through most of a context after its first key."""
    T, hkv = 16384, 1
    n = 64 * torch.cuda.get_device_properties(0).multi_processor_count
    c = Cache(1, hkv, 128, T // 128, code)
    k, v = torch.zeros((1, T, 1, 128), device=DEV), torch.ones((1, T, 1, 128), device=DEV)
    k[:, 0, :, 7] = 240.0
    v[:, 0] = 0.0
    c.append(k.to(dtype), v.to(dtype))
    top = c.held(0, 1)[0][0, 0, 7].item()
    scale = down * float(np.log(2.0)) / top
    q = torch.zeros((1, n, 4, 128), dtype=dtype, device=DEV)
    q[..., 7] = 1.0
    q[:, :, 1::2, 9] = 1.0  # (nothing there: the same scores)
    o = _prefill(c, q, [T - n], T, scale=scale)
    assert o.double().min().item() > 0
    _check(c, q, o, [T - n], [n], scale=scale, rows=64)
    assert c.c.status.item() == 0


def _visible_mean(c, b, pos, g):
    v = c.held(b, pos + 1)[1]
    return v.mean(1).repeat_interleave(g, 0)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("n,start", [(37, 0), (1, 0), (70, 33), (129, 500), (33, 31)])
def test_zero_queries_over_zero_keys_give_the_mean(dtype, code, n, start):
    """Rows of zeros, and rows too small to tell from them, over blocks of zeros: every key counts alike.  Chunks that end
    inside a record of 32 keys, with values and without."""
    T = start + n
    for v in (_tokens(20, (1, T, 2, 128)).to(dtype), torch.zeros((1, T, 2, 128), dtype=dtype, device=DEV)):
        c = Cache(1, 2, 64, 10, code)
        c.append(torch.zeros((1, T, 2, 128), dtype=dtype, device=DEV), v)
        for tiny in (0.0, 1e-30 if dtype == BF16 else 6e-8):
            q = torch.full((1, n, 8, 128), tiny, dtype=dtype, device=DEV)
            o = _prefill(c, q, [start], 640)
            assert torch.isfinite(o).all()
            _check(c, q, o, [start], [n])
            want = _visible_mean(c, 0, T - 1, 4)
            assert ((o[0, -1].double() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -10 * v.double().abs().max()).all()
        assert c.c.status.item() == 0


@pytest.mark.parametrize("dtype,code", [(F16, "s8"), (BF16, "e4m3")])
def test_zero_blocks_among_others(dtype, code):
    """Rows of zeros over keys some of whose blocks are zeros, and ordinary rows beside them."""
    n = 300
    c = Cache(1, 1, 32, 10, code)
    k, v = _tokens(21, (1, n, 1, 128)), _tokens(22, (1, n, 1, 128))
    k[:, 32:96], k[:, 288:] = 0.0, 0.0
    c.append(k.to(dtype), v.to(dtype))
    q = _q(23, (1, n, 4, 128), dtype)
    q[:, ::3] = 0.0
    q[:, 1::7, 2] = 0.0
    o = _prefill(c, q, [0], 320)
    _check(c, q, o, [0], [n], rows=300)
    assert c.c.status.item() == 0


def _check_local(cache, q, o, pos0, scale, rows, gone=None, b=0):
    """As _check, with what the rows really meet in the place of vtop: a key is off by 2^-32 of the largest weight times
    largest |V| of a block."""
    n = q.shape[1]
    T = pos0 + n
    k, v = cache.held(b, T)
    there = torch.ones(T, dtype=torch.bool, device=DEV) if gone is None else ~gone[:T].to(DEV)
    k[:, ~there], v[:, ~there] = 0.0, 0.0
    pad = -T % 32
    top = torch.nn.functional.pad(v.abs().amax(2), (0, pad)).view(cache.hkv, -1, 32).amax(2).repeat_interleave(32, 1)[:, :T]
    g = q.shape[2] // cache.hkv
    k, v, top = (x.repeat_interleave(g, 0) for x in (k, v, top))
    used = 0.0
    for i in sorted({0, n - 1, *np.linspace(0, n - 1, rows).astype(int).tolist()}):
        x = q[b, i].double()
        see = there & (torch.arange(T, device=DEV) <= pos0 + i)
        w = torch.softmax((scale * torch.einsum("htd,hd->ht", k, x)).masked_fill(~see, float("-inf")), dim=1)
        want, mass = torch.einsum("ht,htd->hd", w, v), torch.einsum("ht,htd->hd", w, v.abs())
        es = np.log2(np.e) * scale * torch.einsum("htd,hd->ht", k.abs(), x.abs()).masked_fill(~see, 0.0).amax(1)[:, None]
        es = es * (2.0 ** -22 + 132 * 2.0 ** -24)
        tol = mass * (1.5 * es + 2.0 ** -20 + T * 2.0 ** -24 + 2.0 ** -11) + T * 2.0 ** -32 * (w * top).amax(1)[:, None]
        tol = tol + want.abs() * HALF_STEP[q.dtype] + (2.0 ** -25 if q.dtype == F16 else 0.0)
        got = o[b, i].double()
        assert torch.isfinite(got).all(), i
        share = ((got - want).abs() / tol.clamp_min(1e-300)).max().item()
        assert share <= 1.0, (i, share)
        used = max(used, share)
    return used


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("missing", [True, False])
def test_parts_of_a_row_whose_scales_are_far_apart(code, missing):
    """One step of 128 keys to a CTA: a part whose first block is zeros and whose others are not; and one whose blocks are
    zeros but count, behind a block of values whose keys count for little (and, missing, one whose first block is not there).
    Neither part's share of the row's sum is lost where they are merged."""
    T, n = 1024, 8
    c = Cache(1, 1, 32, T // 32, code, seed=3)
    k, v = 0.02 * _tokens(30, (1, T, 1, 128)), _tokens(31, (1, T, 1, 128))
    k[..., 9] = 0.0
    v[:, 128:160] = 0.0
    v[:, 512:640] = 0.0
    k[:, 512:544, :, 9] = -600.0
    v[:, 512:544] = _tokens(32, (1, 32, 1, 128))
    gone = torch.zeros(T, dtype=torch.bool)
    if missing:
        v[:, 640:768] = 0.0
        gone[640:672] = True
    c.append(k.to(BF16), v.to(BF16))
    q = 0.3 * _q(33, (1, n, 4, 128), BF16)
    q[..., 9] = 1.0
    keep = c.table.clone()
    if missing:
        c.table[0, 20] = -1
    o = _prefill(c, q, [T - n], T)
    assert c.c.status.item() == (B.IQ_DEVERR_PAGE if missing else 0)
    c.table.copy_(keep)
    _check_local(c, q, o, T - n, 128 ** -0.5, n, gone)


def test_first_blocks_missing_and_blocks_of_zeros():
    """Runs of four steps a CTA: some whose first step has no record and whose others are zeros, some that begin with zeros
    and end with values.  What the zeros weigh stays in the row's sum."""
    T, n, hkv = 9600, 8, 8
    c = Cache(1, hkv, 32, T // 32, "e4m3", seed=4)
    k, v = 0.1 * _tokens(34, (1, T, hkv, 128)), _tokens(35, (1, T, hkv, 128))
    v[:, 256:1536], v[:, 3840:7680] = 0.0, 0.0
    c.append(k.to(BF16), v.to(BF16))
    lost = torch.rand(T // 128, generator=torch.Generator().manual_seed(5)) < 0.5
    lost[6:20] = False  # (here the first zeros end)
    lost = lost.repeat_interleave(4)
    q = _q(36, (1, n, 2 * hkv, 128), BF16)
    keep = c.table.clone()
    c.table[0, lost.to(DEV)] = -1
    o = _prefill(c, q, [T - n], T)
    assert c.c.status.item() == B.IQ_DEVERR_PAGE
    c.table.copy_(keep)
    _check_local(c, q, o, T - n, 128 ** -0.5, n, lost.repeat_interleave(32))


@pytest.mark.parametrize("code", ["e4m3", "s8"])
def test_sums_of_keys_whose_values_are_2_to_the_103_smaller(code):
    """A first block of V's 2^103 larger than the rest, whose keys weigh 2^-120 of theirs, in a run of hundreds of steps:
    the sums, in units of the first block's scale, stay finite."""
    T = 98304
    n = 64 * torch.cuda.get_device_properties(0).multi_processor_count
    c = Cache(1, 1, 128, T // 128, code, seed=6)
    k, v = torch.zeros((1, T, 1, 128), device=DEV), (1.0 + _q(37, (1, T, 1, 128), F32).abs()) * 2.0 ** -50
    v[:, :32] *= 2.0 ** 103
    k[:, :32, :, 7] = -240.0
    k[:, 64:, :, 8] = 8.0
    c.append(k.to(BF16), v.to(BF16))
    top = -c.held(0, 1)[0][0, 0, 7].item()
    scale = 120 * float(np.log(2.0)) / top
    q = torch.zeros((1, n, 4, 128), dtype=BF16, device=DEV)
    q[..., 7] = 1.0
    q[..., 8] = 0.475  # the later keys 2^1.9 above the first ones: the probabilities of a half-step just below their limit
    o = _prefill(c, q, [T - n], T, scale=scale)
    assert c.c.status.item() == 0
    _check_local(c, q, o, T - n, scale, 24)


def test_a_million_keys_of_the_smallest_values():
    T, n = 1 << 20, 4
    c = Cache(1, 1, 256, T // 256, "e4m3", seed=7)
    v = _q(38, (1, T, 1, 128), BF16) * 2.0 ** -97 + 2.0 ** -98
    c.append(_q(39, (1, T, 1, 128), BF16), v)
    del v
    q = 0.1 * _q(40, (1, n, 1, 128), BF16)
    o = _prefill(c, q, [T - n], T)
    assert c.c.status.item() == 0 and o.double().abs().max().item() > 0
    _check_local(c, q, o, T - n, 128 ** -0.5, 2)
