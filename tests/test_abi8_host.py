"""Host-side checks of the 8-bit cache's, rotary positions' and pages' entry points: refusals before any launch,
host-only calls, and what the binding refuses of tensors."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import rope
from rotated_bit_kv_iq_b200 import binding as B

cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")


@pytest.fixture(scope="module")
def lib():
    from rotated_bit_kv_iq_b200 import build

    build.build()
    return B.lib()


def _cache(**kw):
    c = B.iq_cache8(0x10000, 2, 2, 128, 64, 4, None, 1, None, B.IQ_E4M3)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(head_dim=64), B.IQ_ERR_UNSUPPORTED), (dict(page_size=24), B.IQ_ERR_INVALID_ARG),
              (dict(pool=None), B.IQ_ERR_INVALID_ARG), (dict(pool=0x10008), B.IQ_ERR_ALIGNMENT),
              (dict(code=2), B.IQ_ERR_UNSUPPORTED), (dict(code=-1), B.IQ_ERR_UNSUPPORTED),
              (dict(n_layers=0), B.IQ_ERR_INVALID_ARG), (dict(status_dev=0x10001), B.IQ_ERR_ALIGNMENT),
              (dict(block_table_dev=0xB0000, max_pages_per_seq=0), B.IQ_ERR_INVALID_ARG)]


def test_library_exports_every_declared_symbol(lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    hdr = open(os.path.join(root, "include", "iq8.h")).read()
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(iq_\w+)\s*\(", hdr, flags=re.M))
    assert len(names) == 15
    for n in names:
        assert hasattr(lib, n) and hasattr(B, n) or n == "iq_pages_workspace_size", n


def test_cache8_bytes(lib):
    assert B.iq_cache8_bytes(2, 4, 64, 10) == 2 * 4 * 64 * 10 * 257
    for bad in ((0, 1, 64, 1), (1, 1, 48, 1), (1, 1, 64, 0), (1, 0, 64, 1)):
        with pytest.raises(B.IqError):
            B.iq_cache8_bytes(*bad)


@cpu_only
def test_append8_rejects_bad_arguments(lib):
    def f(c, layer=0, k=0x50000, v=0x60000, dtype=0, ks=0, vs=0, batch=1, n=4, start=0x70000, valid=None):
        return lib.iq_append8(ctypes.byref(c) if c is not None else None, layer, k, v, dtype, ks, vs, batch, n, start,
                              valid, None)

    assert f(None) == B.IQ_ERR_INVALID_ARG
    for kw, want in BAD_CACHES:
        assert f(_cache(**kw)) == want, kw
    for kw, want in ((dict(layer=2), 1), (dict(k=None, v=None), 1), (dict(start=None), 1), (dict(dtype=3), 2),
                     (dict(ks=128), 1), (dict(vs=260), 1), (dict(n=65), 3), (dict(batch=5), 3), (dict(n=-1), 1),
                     (dict(k=0x50008), 5), (dict(valid=0x50002), 5), (dict(batch=-1), 1)):
        assert f(_cache(), **kw) == want, kw


@cpu_only
def test_attention8_rejects_bad_arguments(lib):
    def dec(c, layer=0, q=0x50000, dtype=0, batch=1, hq=8, ctx=0x70000, max_ctx=32, scale=0.1, out=0x90000, ws=0xA0000,
            ws_bytes=1 << 30):
        return lib.iq_decode8_attention(ctypes.byref(c) if c is not None else None, layer, q, dtype, batch, hq, ctx,
                                        max_ctx, scale, out, ws, ws_bytes, None)

    def pre(c, layer=0, q=0x50000, dtype=0, batch=1, n=8, hq=8, ctx=0x70000, valid=None, max_ctx=32, scale=0.1,
            out=0x90000, ws=0xA0000, ws_bytes=1 << 30):
        return lib.iq_prefill8_attention(ctypes.byref(c) if c is not None else None, layer, q, dtype, batch, n, hq, ctx,
                                         valid, max_ctx, scale, out, ws, ws_bytes, None)

    common = [(dict(layer=-1), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(ctx=None), 1), (dict(dtype=3), 2),
              (dict(hq=18), 2), (dict(hq=5), 1), (dict(hq=0), 1), (dict(max_ctx=65), 3), (dict(batch=5), 3),
              (dict(batch=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
              (dict(scale=float("inf")), 1), (dict(q=0x50004), 5), (dict(out=0x90008), 5), (dict(ws=None), 4),
              (dict(ws_bytes=16), 4), (dict(ws=0xA0010), 5)]
    for f in (dec, pre):
        assert f(None) == B.IQ_ERR_INVALID_ARG
        for kw, want in BAD_CACHES:
            assert f(_cache(**kw)) == want, kw
        for kw, want in common:
            assert f(_cache(), **kw) == want, (f.__name__, kw)
    assert dec(_cache(block_table_dev=0xB0000, max_pages_per_seq=1), batch=2049) == B.IQ_ERR_UNSUPPORTED
    assert dec(_cache(), max_ctx=-1) == B.IQ_ERR_INVALID_ARG
    # lengths that tiles or steps of 32 bits could not count
    far = dict(block_table_dev=0xB0000, page_size=1 << 20, max_pages_per_seq=2047)
    assert dec(_cache(**far), max_ctx=(1 << 30) + 1) == B.IQ_ERR_UNSUPPORTED
    assert dec(_cache(n_kv_heads=64, **far), hq=64, max_ctx=(1 << 29) + 1) == B.IQ_ERR_UNSUPPORTED
    assert pre(_cache(**far), max_ctx=(1 << 30) + 1) == B.IQ_ERR_UNSUPPORTED
    assert pre(_cache(**far), batch=64, n=64 * 64, max_ctx=1 << 28) == B.IQ_ERR_UNSUPPORTED
    assert pre(_cache(**far), batch=64, n=(1 << 20) + 1, max_ctx=1 << 21) == B.IQ_ERR_UNSUPPORTED
    assert pre(_cache(), n=33) == B.IQ_ERR_INVALID_ARG  # max_ctx below the chunk
    assert pre(_cache(), valid=0x70002) == B.IQ_ERR_ALIGNMENT
    assert B.iq_decode8_workspace_size(1, 8, 0, 10) == 0 and B.iq_prefill8_workspace_size(1, 1, 1, 2, 10) == 0


@cpu_only
def test_export8_rejects_bad_arguments(lib):
    f = lib.iq_export8
    c = ctypes.byref(_cache())
    assert f(c, 0, 2, 0, 0, 4, 0x50000, None) == 1 and f(c, 0, 0, 4, 0, 4, 0x50000, None) == 3
    assert f(c, 0, 0, 0, 60, 8, 0x50000, None) == 3 and f(c, 0, 0, 0, 0, 4, None, None) == 1


@cpu_only
def test_rope_rejects_bad_arguments(lib):
    def f(q=0x10000, qs=0, qo=0x20000, qos=0, k=0x30000, ks=0, ko=0x40000, kos=0, dtype=0, n=4, hq=4, hk=2, rd=64,
          layout=0, pos=0x50000, freq=0x60000, ms=1.0):
        return lib.iq_rope(q, qs, qo, qos, k, ks, ko, kos, dtype, n, hq, hk, rd, layout, pos, freq, ms, 0, None)

    for kw, want in ((dict(q=None), 1), (dict(q=None, qo=None, k=None, ko=None), 1), (dict(ko=None), 1), (dict(n=-1), 1),
                     (dict(pos=None), 1), (dict(freq=None), 1), (dict(hq=0), 1), (dict(dtype=3), 2), (dict(layout=2), 2),
                     (dict(rd=0), 2), (dict(rd=63), 2), (dict(rd=130), 2), (dict(qs=256), 1), (dict(qs=516), 1),
                     (dict(qo=0x10000, qs=512, qos=1024), 1), (dict(q=0x10008), 5), (dict(freq=0x60004), 5),
                     (dict(ms=float("nan")), 1)):
        assert f(**kw) == want, kw


@cpu_only
def test_pages_reject_bad_arguments(lib):
    good = dict(block_table_dev=0x10000, seq_len_dev=0x20000, ref_dev=0x30000, max_seqs=4, max_pages_per_seq=3,
                page_size=64, n_pages=9, status_dev=None)

    def p(**kw):
        return ctypes.byref(B.iq_pages(**{**good, **kw}))

    pool = (B.iq_page_pool * 1)(B.iq_page_pool(0x100000, 1, 1, 3200))
    ws, big = 0xA0000, 1 << 30
    calls = {
        "extend": lambda t, a=0x40000, b=0x50000, n=2, w=ws, m=big: lib.iq_pages_extend(t, a, b, n, w, m, None),
        "fork": lambda t, a=0x40000, b=0x50000, n=2, w=ws, m=big: lib.iq_pages_fork(t, pool, 1, a, b, n, w, m, None),
        "copy": lambda t, a=0x40000, b=0x50000, n=2, w=ws, m=big: lib.iq_pages_copy(t, pool, 1, a, b, n, w, m, None),
        "free": lambda t, a=0x40000, b=0x50000, n=2, w=ws, m=big: lib.iq_pages_free(t, a, n, None),
        "compact": lambda t, a=0x40000, b=0x50000, n=2, w=ws, m=big: lib.iq_pages_compact(t, pool, 1, None, w, m, None),
    }
    for name, f in calls.items():
        assert f(None) == 1, name
        for kw, want in ((dict(block_table_dev=None), 1), (dict(ref_dev=None), 1), (dict(max_seqs=0), 1),
                         (dict(page_size=48), 1), (dict(n_pages=0), 1), (dict(seq_len_dev=0x20002), 5)):
            assert f(p(**kw)) == want, (name, kw)
        if name != "compact":
            assert f(p(), a=None) == 1 and f(p(), n=-1) == 1 and f(p(), n=4097) == 2 and f(p(), a=0x40002) == 5, name
        if name not in ("free",):
            assert f(p(), w=None) == 4 and f(p(), m=64) == 4 and f(p(), w=0xA0080) == 5, name
    for bad, want in ((B.iq_page_pool(None, 1, 1, 3200), 1), (B.iq_page_pool(0x100000, 0, 1, 3200), 1),
                      (B.iq_page_pool(0x100000, 1, 1, 24), 1), (B.iq_page_pool(0x100008, 1, 1, 3200), 5)):
        one = (B.iq_page_pool * 1)(bad)
        assert lib.iq_pages_compact(p(), one, 1, None, ws, big, None) == want
    assert lib.iq_pages_compact(p(), pool, 9, None, ws, big, None) == 1
    assert lib.iq_pages_workspace_size(p(n_pages=0)) == 0 and lib.iq_pages_workspace_size(p()) > 0


@pytest.mark.parametrize("scaling", ["plain", "linear", "ntk", "bands", "yarn"])
@pytest.mark.parametrize("rd,base", [(128, 10000.0), (64, 500000.0), (6, 10000.0)])
def test_rope_frequencies_match_the_oracle(lib, scaling, rd, base):
    f, ms = B.iq_rope_frequencies(rd, base, scaling, 8.0, 8192.0, 1.0, 32.0)
    g, want = rope.frequencies(rd, base, scaling, 8.0, 8192.0, 1.0, 32.0)
    np.testing.assert_allclose(f, g, rtol=1e-13)  # a few roundings of 2^-53 in pow and log
    assert abs(ms - want) < 1e-15


def test_rope_frequencies_refusals(lib):
    for a in ((0, 1e4), (63, 1e4), (130, 1e4), (64, 1.0), (64, float("nan")), (64, 1e4, "linear", 0.5), (2, 1e4, "ntk", 2.0),
              (64, 1e4, "bands", 8.0, 0.0), (64, 1e4, "yarn", 8.0, 8192.0, 32.0, 1.0), (64, 1e4, 5)):
        with pytest.raises(B.IqError):
            B.iq_rope_frequencies(*a)


def test_binding_refuses_tensors_of_another_device_shape_or_type(lib):
    """On the CPU: tensors that are not on a GPU are refused before any call."""
    with pytest.raises(ValueError):
        B.PagedCache8(1, 1, 32, 1, pool=torch.zeros(8223, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.PagedCache8(1, 1, 32, 1, pool=torch.zeros(8224, dtype=torch.int8))
    with pytest.raises(ValueError):
        B.PageTable(2, 3, 64, 5, device="cpu", seq_len=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.PageTable(2, 3, 48, 5, device="cpu")
    with pytest.raises(ValueError):
        B.iq_rope(None, None, torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))
    c = B.PagedCache8(1, 2, 32, 1, device="cpu")
    k = torch.zeros(1, 3, 2, 128, dtype=torch.float16)
    s = torch.zeros(1, dtype=torch.int32)
    for kk, ss in ((k.transpose(1, 2), s), (k.to(torch.float64), s), (k[..., :64], s), (k, s.long()), (k, s.repeat(2)),
                   (k.repeat(2, 1, 1, 1), s.repeat(2))):
        with pytest.raises(ValueError):
            B.iq_append8(c, 0, kk, None, ss)
    q = torch.zeros(1, 4, 128)
    w = torch.zeros(1 << 20, dtype=torch.uint8)
    for qq, oo in ((q.half(), q), (q, q[:, :2]), (q.transpose(0, 1), q.transpose(0, 1)), (q.double(), q.double())):
        with pytest.raises(ValueError):
            B.iq_decode8_attention(c, 0, qq, s, 32, oo, w)
    with pytest.raises(ValueError):
        B.iq_append8(c, 0, k, None, s)  # nothing wrong but the device


def test_binding_refuses_broadcast_rows(lib):
    """Rows that share their memory have a stride of 0, which would be taken for the default."""
    c = B.PagedCache8(1, 2, 32, 4, device="cpu")
    for k in (torch.zeros(1, 1, 2, 128).expand(1, 3, 2, 128), torch.zeros(1, 1, 2, 128).expand(3, 1, 2, 128),
              torch.zeros(1, 1, 2, 128).expand(2, 4, 2, 128), torch.zeros(3, 2, 128)):
        with pytest.raises(ValueError, match="wanted") as e:
            B.iq_append8(c, 0, k, None, torch.zeros(k.shape[0], dtype=torch.int32))
        assert "CUDA tensors wanted" not in str(e.value)
    x, y = torch.zeros(1, 2, 128).expand(4, 2, 128), torch.zeros(4, 2, 128)
    pos, freq = torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.float64)
    for q, o in ((x, y), (y, x), (x, None), (torch.zeros(128), None)):
        with pytest.raises(ValueError, match="wanted") as e:
            B.iq_rope(q, None, pos, freq, q_out=o)
        assert "CUDA tensors wanted" not in str(e.value)
