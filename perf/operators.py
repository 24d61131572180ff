"""Cases of the operators around an 8-bit paged KV cache: rotary positions of q and k, quantise-and-append,
decode and prefill attention over the cache, and the operations on its pages.

Where ``own`` is false, run() computes them from elementary torch operations; where it is true, run() makes the
calls of rotated_bit_kv_iq_b200.binding."""

import math
import random

import torch

own = False

D = 128           # head dimension
TT = 32           # tokens of a tile record: one scale for its K, one for its V
TB8 = 8224        # bytes of an 8-bit tile record: K rows, V rows, two float32 scales, 24 spare bytes
TB3 = 3200        # bytes of a 3-bit packed tile record (pages of either cache move the same way)
DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of 16 sequences, 32 query and 8 kv heads, rotated before the append: a latency call.
        dict(name="rope_step", op="rope", tokens=16, hq=32, hkv=8, dtype="f16", layout="half", rd=128, base=500000.0,
             factor=1.0, far=32768, inverse=False),
        # A prompt of 8192 tokens, half of each head rotated in neighbouring pairs, frequencies stretched fourfold.
        dict(name="rope_prompt", op="rope", tokens=8192, hq=32, hkv=8, dtype="bf16", layout="interleaved", rd=64,
             base=10000.0, factor=4.0, far=131072, inverse=False),
        # The new token of each of 16 paged sequences, at whatever slot of its tile it falls.
        dict(name="append_step", op="append", batch=16, n=1, hkv=8, dtype="f16", code="e4m3", page=64, cap=2048,
             lens=1, ragged=False),
        # A 32K prompt of one sequence (the ingest workload's layer) into a contiguous cache.
        dict(name="append_prompt", op="append", batch=1, n=32768, hkv=8, dtype="bf16", code="s8", page=32768, cap=32768,
             lens=0, ragged=False),
        # The smallest decode call: one short sequence, float32 queries.
        dict(name="decode_short", op="decode", batch=1, hq=8, hkv=2, lo=512, hi=512, page=512, dtype="f32", code="e4m3",
             lens=0),
        # One layer of a single 32K sequence with 32 query and 4 kv heads: everything is split over the context.
        dict(name="decode_long", op="decode", batch=1, hq=32, hkv=4, lo=32768, hi=32768, page=32768, dtype="bf16",
             code="s8", lens=0),
        # One layer of the serving workload: 16 ragged sequences of 2K to 32K on shuffled 64-token pages.
        dict(name="decode_serve", op="decode", batch=16, hq=32, hkv=8, lo=2048, hi=32768, page=64, dtype="f16",
             code="e4m3", lens=4),
        # A padded batch of short chunks of odd lengths (one of them empty) at odd positions, float32 queries.
        dict(name="prefill_ragged", op="prefill", batch=4, n=33, hq=12, hkv=2, far=500, page=64, dtype="f32",
             code="e4m3", lens=3, ragged=True),
        # The last 512-token chunk of an 8192-token prompt, 32 query and 8 kv heads.
        dict(name="prefill_chunk", op="prefill", batch=1, n=512, hq=32, hkv=8, far=7680, page=64, dtype="f16",
             code="e4m3", lens=-1, ragged=False),
        # A long chunk: 2048 tokens after 6144.
        dict(name="prefill_long", op="prefill", batch=1, n=2048, hq=32, hkv=8, far=6144, page=64, dtype="bf16",
             code="s8", lens=-1, ragged=False),
        # A beam step on the 3-bit cache: eight losing beams leave, eight winners are forked (their last, part-filled
        # pages copied in all 32 layers).
        dict(name="pages_beams", op="fork", n=8, layers=32, hkv=8, page=64, tb=TB3, lo=700, hi=1500, lens=2),
        # A scheduler's turn on the 8-bit cache: a batch of finished sequences leaves, the pool closes up, a new batch
        # gets its pages.
        dict(name="pages_churn", op="churn", groups=4, n=4, layers=8, hkv=8, page=64, tb=TB8, lo=1000, hi=3000, lens=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "prefill", "prefill", "fork", "churn"])
    hkv, g = rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 6000), hq=min(32, hkv * g), hkv=hkv, dtype=rng.choice(sorted(DTYPES)),
                    layout=rng.choice(["half", "interleaved"]), rd=2 * rng.choice([1, 5, 16, 20, 32, 37, 48, 64, 64]),
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 8.0]), far=_log(rng, 64, 1 << 20),
                    inverse=rng.random() < 0.3)
    dtype, code = rng.choice(sorted(DTYPES)), rng.choice(["e4m3", "s8"])
    page = rng.choice([32, 64, 96, 128])
    lens = rng.randrange(1 << 20)
    if op == "append":
        batch = _log(rng, 1, 32)
        n = rng.choice([1, 1, _log(rng, 2, max(3, 8192 // batch))])
        return dict(op=op, batch=batch, n=n, hkv=hkv, dtype=dtype, code=code, page=page, cap=n + _log(rng, 32, 1024),
                    lens=lens, ragged=rng.random() < 0.5)
    if op == "decode":
        batch = _log(rng, 1, 16)
        hi = _log(rng, 1, min(24000, 200000 // batch))
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, lo=rng.choice([0, hi // 2]), hi=hi, page=page, dtype=dtype,
                    code=code, lens=lens)
    if op == "prefill":
        batch = rng.choice([1, 2, 4])
        hkv, g = rng.choice([1, 2, 4]), rng.randint(1, 8)
        return dict(op=op, batch=batch, n=_log(rng, 1, 1600 // batch), hq=hkv * g, hkv=hkv, far=_log(rng, 1, 6000), page=page,
                    dtype=dtype, code=code, lens=lens, ragged=rng.random() < 0.5)
    tb = rng.choice([TB3, TB8])
    layers = _log(rng, 1, 8)
    hi = _log(rng, 40, 2000)
    n = _log(rng, 1, 12)
    if op == "fork":
        return dict(op=op, n=n, layers=layers, hkv=hkv, page=page, tb=tb, lo=rng.choice([0, hi // 2]), hi=hi, lens=lens)
    return dict(op=op, groups=rng.randint(2, 4), n=min(n, 4), layers=layers, hkv=min(hkv, 4), page=page, tb=tb, lo=1,
                hi=hi, lens=lens)


def _lengths(case, n, lo, hi, salt=0):
    """n whole numbers in [lo, hi], fixed by the case."""
    r = random.Random(case["lens"] * 8 + salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _plan(case):
    """The lengths that the case fixes: per sequence."""
    if case["op"] == "append":
        cnt = [case["n"]] * case["batch"]
        if case["ragged"]:
            cnt[1:] = _lengths(case, case["batch"] - 1, 0, case["n"], 1)
        return [s % (case["cap"] - case["n"] + 1) for s in _lengths(case, case["batch"], 0, case["cap"])], cnt
    if case["op"] == "decode":
        return _lengths(case, case["batch"], case["lo"], case["hi"])
    if case["op"] == "prefill":
        far = case["far"]
        start = [far] * case["batch"] if case["lens"] < 0 else _lengths(case, case["batch"], 0, far)
        cnt = [case["n"]] * case["batch"]
        if case["ragged"]:
            cnt = [case["n"], 1, 0, case["n"] // 2][: case["batch"]]
        return start, cnt
    if case["op"] == "fork":
        return _lengths(case, case["n"], case["lo"], case["hi"]), [
            p % case["n"] for p in _lengths(case, case["n"], 0, 1 << 20, 1)]
    return _lengths(case, case["n"], case["lo"], case["hi"])


def work(case):
    op = case["op"]
    if op == "rope":
        v = case["tokens"] * (case["hq"] + case["hkv"]) * D
        return {"bytes": 2 * v * DTYPES[case["dtype"]].itemsize + 4 * case["tokens"], "flops": 3 * v}
    if op == "append":
        t = sum(_plan(case)[1]) * case["hkv"]
        return {"bytes": 2 * t * D * DTYPES[case["dtype"]].itemsize + 257 * t, "flops": 4 * t * D}
    if op == "decode":
        t = sum(_plan(case))
        return {"bytes": 257 * t * case["hkv"] + 2 * case["batch"] * case["hq"] * D * DTYPES[case["dtype"]].itemsize,
                "flops": 4 * D * case["hq"] * t}
    if op == "prefill":
        start, cnt = _plan(case)
        pairs = sum(n * s + n * (n + 1) // 2 for s, n in zip(start, cnt))
        e = DTYPES[case["dtype"]].itemsize
        return {"bytes": 257 * case["hkv"] * sum(s + n for s, n in zip(start, cnt) if n) + 2 * sum(cnt) * case["hq"] * D * e,
                "flops": 4 * D * case["hq"] * pairs}
    per = -(-case["hi"] // case["page"])
    if op == "fork":
        lens, parent = _plan(case)
        tiles = sum(-(-(lens[p] % case["page"]) // TT) for p in parent)
        return {"bytes": 2 * tiles * case["layers"] * case["hkv"] * case["tb"] + 12 * case["n"] * per, "flops": 0}
    pages = sum(-(-x // case["page"]) for x in _plan(case))
    one = case["hkv"] * (case["page"] // TT) * case["tb"]
    return {"bytes": 2 * pages * case["layers"] * one + 8 * case["groups"] * case["n"] * per, "flops": 0}


# ---------------------------------------------------------------------------------------------- inputs
def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed((seed * 1000003 + salt) & 0x7FFFFFFFFFFF)


def _tokens(g, shape):
    """Keys or values as a model makes them: channel scales of their own and four outlying channels a head."""
    hkv = shape[-2]
    s = torch.exp(0.5 * torch.randn((hkv, D), generator=g, device=DEV))
    s.scatter_(1, torch.rand((hkv, D), generator=g, device=DEV).topk(4, dim=1).indices, 12.0)
    return (torch.randn(shape, generator=g, device=DEV) * s).clamp_(-65504.0, 65504.0)


def _swizzle():
    """[32][8]: where the 16-byte chunk c of row s is stored (and, the other way round, which one is stored at c)."""
    s = torch.arange(TT, device=DEV)[:, None]
    return s, torch.arange(8, device=DEV)[None, :] ^ (s & 7)


def _quantise(x, scale, code):
    """Codes (as bytes) of x, shape [..., 32, 128], under scale, shape [...]."""
    y = x / scale[..., None, None]
    if code == "e4m3":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(y).clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _scale_of(amax, code):
    """The scale that largest magnitudes ask for (float32, the same in 32 bits and in 64)."""
    if code == "e4m3":
        m, e = torch.frexp(amax)
        e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-100, 120)
        return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -100))
    bits = (amax / 127.0).clamp_min(2.0 ** -100).view(torch.int32)
    return ((bits + 0xFFFF) & -65536).view(torch.float32)


def _values(rec, code):
    """Tile records [..., 8224] -> K and V values, each [..., 32, 128] float32 (un-swizzled, scaled)."""
    s, at = _swizzle()
    kind = torch.float8_e4m3fn if code == "e4m3" else torch.int8
    x = rec[..., : 2 * TT * D].contiguous().view(kind).float().view(*rec.shape[:-1], 2, TT, 8, 16)[..., s, at, :]
    sc = rec[..., 2 * TT * D: 2 * TT * D + 8].contiguous().view(torch.float32)
    x = x.reshape(*rec.shape[:-1], 2, TT, D) * sc[..., None, None]
    return x[..., 0, :, :], x[..., 1, :, :]


def _cache(case, seed, batch, cap, lens):
    """A filled one-layer 8-bit cache: (pool [1][pages][hkv][tiles][8224], table [batch][per] on shuffled pages). What lies
    behind a sequence's last token is what the memory held: here NaN codes and NaN scales."""
    hkv, page = case["hkv"], case["page"]
    per = max(1, -(-cap // page))
    g = _gen(seed, 1)
    table = torch.randperm(batch * per, generator=g, device=DEV).to(torch.int32).view(batch, per)
    tiles = page // TT
    pool = torch.full((1, batch * per, hkv, tiles, TB8), 0x7F, dtype=torch.uint8, device=DEV)
    pool[..., 2 * TT * D: 2 * TT * D + 8].view(torch.float32).fill_(float("nan"))
    s, at = _swizzle()
    ln = torch.tensor(lens, device=DEV)
    pos = torch.arange(per * page, device=DEV).view(per, tiles, TT)
    live = pos < ln.view(-1, 1, 1, 1)  # [batch][per][tiles][32]
    for side in (0, 1):
        x = _tokens(g, (batch, per, tiles, TT, hkv, D)).permute(0, 1, 4, 2, 3, 5)  # [batch][per][hkv][tiles][32][128]
        m = live[:, :, None, :, :, None]
        scale = _scale_of(torch.where(m, x.abs(), 0.0).amax((-1, -2)), case["code"])
        c = torch.where(m, _quantise(x, scale, case["code"]), 0x7F).reshape(batch, per, hkv, tiles, TT, 8, 16)
        rows = pool[0, :, :, :, side * TT * D: (side + 1) * TT * D]
        rows[table.long()] = c[..., s, at, :].reshape(batch, per, hkv, tiles, TT * D)
        sc = pool[0, :, :, :, 2 * TT * D + 4 * side: 2 * TT * D + 4 * side + 4].view(torch.float32)[..., 0]
        sc[table.long()] = torch.where(live.any(-1)[:, :, None, :], scale, float("nan"))
        del x, c
    return pool, table


def prepare(case, seed):
    op, st = case["op"], {"case": case}
    if own:
        from rotated_bit_kv_iq_b200 import binding as B
    if op == "rope":
        g, n = _gen(seed, 2), case["tokens"]
        # q and k as the fused projection leaves them: slices of one row per token
        qkv = torch.randn((n, case["hq"] + 2 * case["hkv"], D), generator=g, device=DEV).to(DTYPES[case["dtype"]])
        st["q"], st["k"] = qkv[:, : case["hq"]], qkv[:, case["hq"]: case["hq"] + case["hkv"]]
        st["pos"] = torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
        st["freq"], st["ms"] = _frequencies(case)
        if own:
            st["out"] = (torch.empty((n, case["hq"], D), dtype=qkv.dtype, device=DEV),
                         torch.empty((n, case["hkv"], D), dtype=qkv.dtype, device=DEV))
    elif op == "append":
        start, cnt = _plan(case)
        st["pool"], st["table"] = _cache(case, seed, case["batch"], case["cap"], start)
        g = _gen(seed, 3)
        shape = (case["batch"], case["n"], case["hkv"], D)
        st["k"], st["v"] = (_tokens(g, shape).to(DTYPES[case["dtype"]]) for _ in range(2))
        st["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        st["cnt"] = torch.tensor(cnt, dtype=torch.int32, device=DEV)
        _clean(st)
    elif op in ("decode", "prefill"):
        g, dt = _gen(seed, 4), DTYPES[case["dtype"]]
        if op == "decode":
            lens = _plan(case)
            shape = (case["batch"], case["hq"], D)
        else:
            start, cnt = _plan(case)
            lens = [s + n for s, n in zip(start, cnt)]
            shape = (case["batch"], case["n"], case["hq"], D)
            st["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
            st["cnt"] = torch.tensor(cnt, dtype=torch.int32, device=DEV)
        cap = max(lens + [1]) if op == "decode" else max(start) + case["n"]
        st["pool"], st["table"] = _cache(case, seed, case["batch"], cap, lens)
        st["max"] = cap
        st["len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["q"] = torch.randn(shape, generator=g, device=DEV).to(dt)
        st["out"] = torch.zeros(shape, dtype=dt, device=DEV)
    else:
        _pages(case, seed, st)
    if own and "table" in st and op in ("append", "decode", "prefill"):
        st["cache"] = B.PagedCache8(1, case["hkv"], case["page"], st["pool"].shape[1], block_table=st["table"],
                                    code=case["code"], pool=st["pool"].view(-1))
        if op == "decode":
            need = B.iq_decode8_workspace_size(case["batch"], case["hq"], case["hkv"], st["max"])
        elif op == "prefill":
            need = B.iq_prefill8_workspace_size(case["batch"], case["n"], case["hq"], case["hkv"], st["max"])
        else:
            need = 0
        st["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    if own and op in ("fork", "churn"):
        st["pt"] = B.PageTable(st["table"].shape[0], st["table"].shape[1], case["page"], st["ref"].numel(),
                               block_table=st["table"], seq_len=st["len"], ref=st["ref"])
        st["pp"] = B.PagePool(st["pool"].view(-1), case["layers"], case["hkv"], case["page"], st["ref"].numel(), case["tb"])
        st["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


def _clean(st):
    """The unwritten part of an append's cache as zeros, so that the whole pool can be compared."""
    pool, case = st["pool"], st["case"]
    sc = pool[..., 2 * TT * D: 2 * TT * D + 8].view(torch.float32)
    none = sc.isnan().all(-1)
    sc.nan_to_num_(0.0)
    pool[none] = 0
    if case["code"] == "e4m3":
        rows = pool[..., : 2 * TT * D]
        rows[rows == 0x7F] = 0x7E


def _frequencies(case):
    """Radians a position, float64 [rd/2], stretched for long contexts between two wavelengths; and the factor on q, k."""
    i = torch.arange(0, case["rd"], 2, dtype=torch.float64, device=DEV) / case["rd"]
    f = case["base"] ** -i
    if case["factor"] == 1.0:
        return f, 1.0
    turns = 8192.0 * f / (2 * math.pi)  # turns within the length that was trained
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / case["factor"] * (1 - keep), 0.1 * math.log(case["factor"]) + 1.0


def _pages(case, seed, st):
    """Sequences on a pool of pages, each page's contents its own."""
    g, page = _gen(seed, 5), case["page"]
    fork = case["op"] == "fork"
    lens, extra = _plan(case) if fork else (_plan(case) * case["groups"], None)
    per = max(1, -(-max(lens + [case["hi"]]) // page))
    rows = 2 * case["n"] if fork else len(lens)
    used = sum(-(-x // page) for x in lens)
    n_pages = used + case["n"] + max(4, used // 4)
    table = torch.full((rows, per), -1, dtype=torch.int32)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist() if fork else range(n_pages)
    at = 0
    for r, x in enumerate(lens):
        k = -(-x // page)
        table[r, :k] = torch.tensor(list(order[at: at + k]), dtype=torch.int32)
        at += k
    ref = torch.zeros(n_pages, dtype=torch.int32)
    ref[table[table >= 0].long()] = 1
    st["table"], st["ref"] = table.to(DEV), ref.to(DEV)
    st["len"] = torch.tensor(lens + [0] * (rows - len(lens)), dtype=torch.int32, device=DEV)
    shape = (case["layers"], n_pages, case["hkv"], page // TT, case["tb"])
    st["pool"] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    st["turn"] = 0
    if fork:
        st["child"] = torch.arange(case["n"], 2 * case["n"], dtype=torch.int32, device=DEV)
        st["parent"] = torch.tensor(extra, dtype=torch.int32, device=DEV)
        _fork_plain(st)  # the beams that the pass lets go of
        st["pool"].copy_(torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8))
    else:
        st["ids"] = [torch.arange(k * case["n"], (k + 1) * case["n"], dtype=torch.int32, device=DEV)
                     for k in range(case["groups"])]
        st["want"] = torch.tensor(lens[: case["n"]], dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------ plain forms
def _rope_plain(st):
    case, rd = st["case"], st["case"]["rd"]
    ang = st["pos"].double()[:, None] * st["freq"]
    c, s = (torch.cos(ang) * st["ms"]).float()[:, None], (torch.sin(ang) * st["ms"]).float()[:, None]
    s = -s if case["inverse"] else s

    def turn(x):
        y = x.float()
        a, b = (y[..., : rd // 2], y[..., rd // 2: rd]) if case["layout"] == "half" else (y[..., 0:rd:2], y[..., 1:rd:2])
        u, v = a * c - b * s, a * s + b * c
        r = torch.cat((u, v), -1) if case["layout"] == "half" else torch.stack((u, v), -1).flatten(-2)
        return torch.cat((r.to(x.dtype), x[..., rd:]), -1)

    return {"q": turn(st["q"]), "k": turn(st["k"])}


def _append_plain(st):
    case, pool = st["case"], st["pool"]
    batch, n, hkv, page = case["batch"], case["n"], case["hkv"], case["page"]
    start, cnt = st["start"].long(), st["cnt"].long()
    J = (n + 2 * TT - 2) // TT
    tile = (start // TT)[:, None] + torch.arange(J, device=DEV)  # [batch][J]
    p = tile[..., None] * TT + torch.arange(TT, device=DEV)      # positions [batch][J][32]
    i = p - start[:, None, None]
    new, old = (i >= 0) & (i < cnt[:, None, None]), i < 0
    b, j = torch.nonzero(new.any(-1), as_tuple=True)             # the tiles that get tokens
    new, old, i = new[b, j], old[b, j], i[b, j].clamp(0, n - 1)
    at = st["table"].long()[b, tile[b, j] * TT // page], (tile[b, j] * TT % page) // TT
    s, sw = _swizzle()
    code = case["code"]
    rec = pool[0][at[0], :, at[1]]                               # [m][hkv][8224]
    vals = _values(rec, code)
    for side, x in ((0, st["k"]), (1, st["v"])):
        x = x[b[:, None], i].float().transpose(1, 2)             # [m][hkv][32][128]
        m = new[:, None, :, None]
        scale = _scale_of(torch.where(m & x.isfinite(), x.abs(), 0.0).amax((-1, -2)), code)
        had = rec[..., 2 * TT * D + 4 * side: 2 * TT * D + 4 * side + 4].contiguous().view(torch.float32)[..., 0]
        scale = torch.where(old.any(-1)[:, None], torch.maximum(scale, had), scale)
        both = torch.where(m, x.nan_to_num(0.0, float("inf"), float("-inf")), vals[side])
        both = _quantise(both, scale, code).reshape(*both.shape[:-1], 8, 16)
        rows = rec[..., side * TT * D: (side + 1) * TT * D].view(*rec.shape[:-1], TT, 8, 16)
        rows.copy_(torch.where((new | old)[:, None, :, None, None], both[..., s, sw, :], rows))
        rec[..., 2 * TT * D + 4 * side: 2 * TT * D + 4 * side + 4] = scale[..., None].contiguous().view(torch.uint8)
    pool[0][at[0], :, at[1]] = rec


def _attend(q, pos, st):
    """q [batch][n][hq][128]; query i of sequence b sees the positions up to pos[b][i] (none where that is negative)."""
    case = st["case"]
    rec = st["pool"][0][st["table"].long()]                      # [batch][per][hkv][tiles][8224]
    k, v = _values(rec, case["code"])
    del rec
    batch, hkv = q.shape[0], case["hkv"]
    g = case["hq"] // hkv
    T = k.shape[1] * case["page"]
    k = k.transpose(1, 2).reshape(batch, hkv, T, D)
    v = v.transpose(1, 2).reshape(batch, hkv, T, D)
    t = torch.arange(T, device=DEV)
    live = (t < st["len"][:, None])[:, None, :, None]
    k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)  # what lies behind the last token is no number
    x = q.float().view(batch, -1, hkv, g, D).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, D)
    s = (x @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))         # [batch][hkv][g*n][T]
    see = (t <= pos[..., None])[:, None, None].expand(-1, hkv, g, -1, -1).reshape(batch, hkv, -1, T)
    s = torch.where(see, s, float("-inf"))
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    o = torch.where(l > 0, (e @ v) / l.clamp_min(1e-30), 0.0)
    return o.view(batch, hkv, g, -1, D).permute(0, 3, 1, 2, 4).reshape(batch, -1, case["hq"], D).to(q.dtype)


def _free_plain(st, ids):
    rows = st["table"][ids.long()].long()
    n = st["ref"].numel()
    held = torch.cat((st["ref"], st["ref"].new_zeros(1)))
    held.index_add_(0, torch.where(rows >= 0, rows, n).flatten(), torch.full_like(rows.flatten(), -1, dtype=torch.int32))
    st["ref"].copy_(held[:n])
    st["table"][ids.long()] = -1
    st["len"][ids.long()] = 0


def _fork_plain(st):
    case, page = st["case"], st["case"]["page"]
    ref, parent, child = st["ref"], st["parent"].long(), st["child"].long()
    ln, rows = st["len"][parent].long(), st["table"][parent].long()
    full, part = ln // page, ln % page
    order = torch.argsort((ref != 0).to(torch.int32), stable=True)      # free pages first, the lowest first
    fresh = order[(torch.cumsum((part > 0).long(), 0) - 1).clamp_min(0)]
    j = torch.arange(rows.shape[1], device=DEV)
    tail = (j == full[:, None]) & (part > 0)[:, None]
    new = torch.where(j < full[:, None], rows, torch.where(tail, fresh[:, None], -1))
    n = ref.numel()
    held = torch.cat((ref, ref.new_zeros(1)))
    held.index_add_(0, torch.where(new >= 0, new, n).flatten(), torch.ones_like(new.flatten(), dtype=torch.int32))
    ref.copy_(held[:n])
    st["table"][child] = new.to(torch.int32)
    st["len"][child] = ln.to(torch.int32)
    k = torch.nonzero(part > 0).flatten()
    src, dst = rows[k, full[k]], fresh[k]
    used = (torch.arange(page // TT, device=DEV) * TT < part[k, None])[None, :, None, :, None]
    st["pool"][:, dst] = torch.where(used, st["pool"][:, src], st["pool"][:, dst])


def _compact_plain(st):
    ref = st["ref"]
    live = ref > 0
    i = torch.arange(ref.numel(), device=DEV)
    count = live.sum()
    hole, mover = torch.nonzero(~live & (i < count)).flatten(), torch.nonzero(live & (i >= count)).flatten()
    st["pool"][:, hole] = st["pool"][:, mover]
    to = i.clone()
    to[mover] = hole
    st["table"].copy_(torch.where(st["table"] >= 0, to[st["table"].clamp_min(0).long()], -1))
    ref[hole] = ref[mover]
    ref[mover] = 0
    return count.to(torch.int32).view(1)


def _extend_plain(st, ids, want):
    page, ref, ids = st["case"]["page"], st["ref"], ids.long()
    have, need = (st["len"][ids].long() + page - 1) // page, (want.long() + page - 1) // page
    j = torch.arange(st["table"].shape[1], device=DEV)
    get = (j >= have[:, None]) & (j < need[:, None])
    order = torch.argsort((ref != 0).to(torch.int32), stable=True)
    k = torch.cumsum(get.flatten().long(), 0).view_as(get) - 1
    fresh = order[k.clamp(0, ref.numel() - 1)]
    st["table"][ids] = torch.where(get, fresh.to(torch.int32), st["table"][ids])
    ref[fresh[get]] = 1
    st["len"][ids] = want


def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        return _run_own(st)
    if op == "rope":
        return _rope_plain(st)
    if op == "append":
        _append_plain(st)
        return _held(st)
    if op == "decode":
        o = _attend(st["q"][:, None], st["len"][:, None].long() - 1, st)
        return o[:, 0]
    if op == "prefill":
        i = torch.arange(case["n"], device=DEV)
        o = _attend(st["q"], st["start"].long()[:, None] + i, st)
        st["out"].copy_(torch.where((i < st["cnt"][:, None])[..., None, None], o, st["out"]))
        return st["out"]
    if op == "fork":
        _free_plain(st, st["child"])
        _fork_plain(st)
        return [st["table"], st["len"], st["ref"], st["pool"]]
    ids = st["ids"][st["turn"] % case["groups"]]
    st["turn"] += 1
    _free_plain(st, ids)
    count = _compact_plain(st)
    _extend_plain(st, ids, st["want"])
    return [st["table"], st["len"], st["ref"], st["pool"], count]


def _held(st):
    """What an append leaves: the codes as the numbers that they are, and their scales."""
    pool = st["pool"]
    kind = torch.float8_e4m3fn if st["case"]["code"] == "e4m3" else torch.int8
    return {"codes": pool[..., : 2 * TT * D].view(kind), "scales": pool[..., 2 * TT * D: 2 * TT * D + 8].view(torch.float32)}


def _run_own(st):
    from rotated_bit_kv_iq_b200 import binding as B

    case, op = st["case"], st["case"]["op"]
    if op == "rope":
        q, k = st["out"]
        B.iq_rope(st["q"], st["k"], st["pos"], st["freq"], q, k, layout=case["layout"], mscale=st["ms"],
                  inverse=case["inverse"])
        return {"q": q, "k": k}
    if op == "append":
        B.iq_append8(st["cache"], 0, st["k"], st["v"], st["start"], n_valid=st["cnt"])
        return _held(st)
    if op == "decode":
        B.iq_decode8_attention(st["cache"], 0, st["q"], st["len"], st["max"], st["out"], st["ws"])
        return st["out"]
    if op == "prefill":
        B.iq_prefill8_attention(st["cache"], 0, st["q"], st["start"], st["max"], st["out"], st["ws"],
                                n_valid=st["cnt"])
        return st["out"]
    pt, pp = st["pt"], st["pp"]
    if op == "fork":
        B.iq_pages_free(pt, st["child"])
        B.iq_pages_fork(pt, pp, st["parent"], st["child"])
        return [st["table"], st["len"], st["ref"], st["pool"]]
    ids = st["ids"][st["turn"] % case["groups"]]
    st["turn"] += 1
    B.iq_pages_free(pt, ids)
    B.iq_pages_compact(pt, pp, st["live"])
    B.iq_pages_extend(pt, ids, st["want"])
    return [st["table"], st["len"], st["ref"], st["pool"], st["live"]]


# ---------------------------------------------------------------------------------- the definition in 64 bits
def _round_e4m3(y):
    """Nearest number of three mantissa bits and exponents -6 .. 8, ties to the even one, ends at 448."""
    a = y.abs().clamp_max(448.0)
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -20))).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return torch.sign(y) * (torch.round(a / step) * step).clamp_max(448.0)


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "churn"):
        return None  # whole numbers alone
    st = prepare(case, seed)
    if op == "rope":
        return _exact_rope(st)
    if op == "append":
        return _exact_append(st)
    return _exact_attention(st)


def _exact_rope(st):
    """Each pair as a complex number times ms * exp(i angle), the angle reduced to a turn before the exponential."""
    case, rd = st["case"], st["case"]["rd"]
    ang = torch.remainder(st["pos"].double()[:, None] * st["freq"], 2 * math.pi)
    ang = -ang if case["inverse"] else ang
    z = torch.polar(torch.full_like(ang, st["ms"]), ang)[:, None]
    out = {}
    for name in ("q", "k"):
        y = st[name].double().clone()
        if case["layout"] == "half":
            w = torch.complex(y[..., : rd // 2], y[..., rd // 2: rd].contiguous()) * z
            y[..., : rd // 2], y[..., rd // 2: rd] = w.real, w.imag
        else:
            w = torch.complex(y[..., 0:rd:2].contiguous(), y[..., 1:rd:2].contiguous()) * z
            y[..., 0:rd:2], y[..., 1:rd:2] = w.real, w.imag
        out[name] = y
    return out


def _exact_append(st):
    """Tile after tile, sequence after sequence, in 64 bits."""
    case, page, code = st["case"], st["case"]["page"], st["case"]["code"]
    start, cnt = _plan(case)
    held = _held(st)
    codes, scales = held["codes"].double(), held["scales"].double()
    s, at = _swizzle()
    table = st["table"].tolist()
    x = [st["k"].double(), st["v"].double()]
    for b in range(case["batch"]):
        p, end = start[b], start[b] + cnt[b]
        while p < end:
            lo, hi = p // TT * TT, min(end, p // TT * TT + TT)
            pg, tile = table[b][p // page], p % page // TT
            for side in (0, 1):
                y = x[side][b, p - start[b]: hi - start[b]].transpose(0, 1)  # [hkv][m][128]
                top = y.abs().amax((-1, -2))
                if code == "e4m3":
                    need = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(-100, 120))
                    need = torch.where(need / 2 * 448.0 >= top, need / 2, need)
                else:
                    u = torch.exp2(torch.floor(torch.log2(top / 127.0)) - 7)
                    need = torch.ceil(top / 127.0 / u) * u
                was = scales[0, pg, :, tile, side].clone()
                now = torch.maximum(need, was) if p > lo else need
                rows = codes[0, pg, :, tile, side * TT * D: (side + 1) * TT * D].view(-1, TT, 8, 16)[:, s, at].reshape(-1, TT, D)
                rows[:, : p - lo] *= (was / now)[:, None, None]
                rows[:, p - lo: hi - lo] = y / now[:, None, None]
                m = rows[:, : hi - lo]
                rows[:, : hi - lo] = _round_e4m3(m) if code == "e4m3" else torch.round(m).clamp(-127, 127)
                rows = rows.reshape(-1, TT, 8, 16)
                codes[0, pg, :, tile, side * TT * D: (side + 1) * TT * D] = rows[:, s, at].reshape(-1, TT * D)
                scales[0, pg, :, tile, side] = now
            p = hi
    return {"codes": codes if code == "e4m3" else None, "scales": scales}


def _exact_attention(st):
    """Head after head, over the tokens that are there and no others."""
    case, page, hkv = st["case"], st["case"]["page"], st["case"]["hkv"]
    g = case["hq"] // hkv
    decode = case["op"] == "decode"
    q = (st["q"][:, None] if decode else st["q"]).double()
    out = torch.zeros_like(q)
    cnt = [1] * case["batch"] if decode else st["cnt"].tolist()
    kind = torch.float8_e4m3fn if case["code"] == "e4m3" else torch.int8
    s, at = _swizzle()
    for b, T in enumerate(st["len"].tolist()):
        n = cnt[b] if T else 0
        if not n:
            continue
        rec = st["pool"][0][st["table"][b, : -(-T // page)].long()]  # [pages][hkv][tiles][8224]
        for h in range(hkv):
            r = rec[:, h].reshape(-1, TB8)
            x = r[:, : 2 * TT * D].contiguous().view(kind).double().view(-1, 2, TT, 8, 16)[:, :, s, at].reshape(-1, 2, TT, D)
            x = x * r[:, 2 * TT * D: 2 * TT * D + 8].contiguous().view(torch.float32).double()[..., None, None]
            k, v = x[:, 0].reshape(-1, D)[:T], x[:, 1].reshape(-1, D)[:T]
            see = torch.arange(T, device=DEV) <= torch.arange(T - n, T, device=DEV)[:, None]
            for e in range(h * g, (h + 1) * g):
                w = q[b, :n, e] @ k.T / math.sqrt(D)
                w = torch.softmax(w.masked_fill(~see, float("-inf")), -1)
                out[b, :n, e] = w @ v
    return out[:, 0] if decode else out
