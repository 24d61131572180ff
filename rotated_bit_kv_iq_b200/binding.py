"""ctypes binding of libiq (include/iq.h, include/iq8.h): argument marshalling only.

Every entry point keeps its C name.  Device buffers are torch CUDA tensors (PyTorch is used
for device memory and streams only); every step of the computation runs in libiq's kernels.
Loading fails loudly when libiq.so is missing: there is no CPU fallback.
"""

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libiq.so")

IQ_OK = 0
IQ_ERR_INVALID_ARG = 1
IQ_ERR_UNSUPPORTED = 2
IQ_ERR_CAPACITY = 3
IQ_ERR_WORKSPACE = 4
IQ_ERR_ALIGNMENT = 5
IQ_ERR_CUDA = 6
IQ_F16 = 0
IQ_F32 = 1
IQ_BF16 = 2  # the calls on the 8-bit cache and iq_rope only
IQ_DEVERR_POSITION = 1
IQ_DEVERR_PAGE = 2
IQ_DEVERR_CTX = 4
IQ_DEVERR_TIMEOUT = 8
IQ_DEVERR_WORKSPACE = 16
IQ_DEVERR_SEQ = 32
IQ_DEVERR_NOPAGE = 64
IQ_DEVERR_RANGE = 128
IQ_ROT_ISO = 0
IQ_ROT_QUAT = 1
IQ_ROT_PLANAR = 2
ROTATIONS = {"iso": IQ_ROT_ISO, "quat": IQ_ROT_QUAT, "planar": IQ_ROT_PLANAR}
WIDTHS = ((2, 2), (3, 2), (3, 3), (4, 2), (4, 3), (4, 4))  # supported (K bits, V bits)

IQ_E4M3 = 0
IQ_S8 = 1
CODES8 = {"e4m3": IQ_E4M3, "s8": IQ_S8}
TILE8_BYTES = 8224
IQ_ROPE_HALF = 0
IQ_ROPE_INTERLEAVED = 1
ROPE_LAYOUTS = {"half": IQ_ROPE_HALF, "interleaved": IQ_ROPE_INTERLEAVED}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}
IQ_PAGES_MAX_LIST = 4096

HEAD_DIM = 128
V_BLOCK_TOKENS = 16
TILE_TOKENS = 32


def k_record_bytes(bits=3):
    return 16 * bits


def v_block_bytes(bits=3):
    return 256 * bits


def tile_bytes(k_bits=3, v_bits=3):
    """32 K records | 2 V blocks | 32 K norms | 32 V norms (3200 bytes for 3/3)."""
    return 32 * k_record_bytes(k_bits) + 2 * v_block_bytes(v_bits) + 128


K_RECORD_BYTES = k_record_bytes(3)
V_BLOCK_BYTES = v_block_bytes(3)
TILE_BYTES = tile_bytes(3, 3)


class IqError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn}: {iq_status_string(status)} (status {status})")
        self.status = status


class iq_cache(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p),
        ("n_layers", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
        ("block_table_dev", ctypes.c_void_p),
        ("max_pages_per_seq", ctypes.c_int32),
        ("status_dev", ctypes.c_void_p),
        ("k_bits", ctypes.c_int32),
        ("v_bits", ctypes.c_int32),
        ("rotation", ctypes.c_int32),
    ]


class iq_fp16_prefix(ctypes.Structure):
    _fields_ = [
        ("k_dev", ctypes.c_void_p),
        ("v_dev", ctypes.c_void_p),
        ("len_dev", ctypes.c_void_p),
        ("max_len", ctypes.c_int32),
    ]


class iq_cache8(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p),
        ("n_layers", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
        ("block_table_dev", ctypes.c_void_p),
        ("max_pages_per_seq", ctypes.c_int32),
        ("status_dev", ctypes.c_void_p),
        ("code", ctypes.c_int32),
    ]


class iq_pages(ctypes.Structure):
    _fields_ = [
        ("block_table_dev", ctypes.c_void_p),
        ("seq_len_dev", ctypes.c_void_p),
        ("ref_dev", ctypes.c_void_p),
        ("max_seqs", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
        ("status_dev", ctypes.c_void_p),
    ]


class iq_page_pool(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p),
        ("n_layers", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("tile_bytes", ctypes.c_int32),
    ]


_lib = None


def lib():
    """Load libiq.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libiq.so not built at {LIB_PATH}; run `python -m rotated_bit_kv_iq_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        P = ctypes.POINTER(iq_cache)
        L.iq_version.restype = ctypes.c_char_p
        L.iq_version.argtypes = []
        L.iq_status_string.restype = ctypes.c_char_p
        L.iq_status_string.argtypes = [ctypes.c_int]
        L.iq_cache_bytes.restype = ctypes.c_int
        L.iq_cache_bytes.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.iq_init_rotation.restype = ctypes.c_int
        L.iq_init_rotation.argtypes = [ctypes.c_uint64, i32, i32, vp]
        L.iq_init_rotation_variant.restype = ctypes.c_int
        L.iq_init_rotation_variant.argtypes = [ctypes.c_uint64, i32, i32, i32, vp]
        L.iq_rotation_params_per_head.restype = i32
        L.iq_rotation_params_per_head.argtypes = [i32]
        L.iq_encode_append.restype = ctypes.c_int
        L.iq_encode_append.argtypes = [P, i32, vp, vp, i32, i32, vp, vp, vp]
        L.iq_decode_workspace_size.restype = sz
        L.iq_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        L.iq_decode_attention.restype = ctypes.c_int
        L.iq_decode_attention.argtypes = [P, i32, vp, ctypes.c_int, i32, i32, vp, i32, vp, vp, vp, sz, vp]
        L.iq_decode_step.restype = ctypes.c_int
        L.iq_decode_step.argtypes = [P, i32, vp, ctypes.c_int, vp, vp, i32, i32, vp, i32, vp, vp, vp, sz, vp]
        L.iq_decode_attention_noalloc.restype = ctypes.c_int
        L.iq_decode_attention_noalloc.argtypes = [P, i32, vp, ctypes.c_int, i32, i32, vp, i32, vp, vp, vp]
        L.iq_decode_deferred_workspace_size.restype = sz
        L.iq_decode_deferred_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.iq_decode_step_deferred.restype = ctypes.c_int
        L.iq_decode_step_deferred.argtypes = [P, i32, ctypes.POINTER(iq_fp16_prefix), vp, ctypes.c_int, vp, vp, i32,
                                              i32, vp, i32, vp, vp, vp, sz, vp]
        L.iq_prefill_workspace_size.restype = sz
        L.iq_prefill_workspace_size.argtypes = [i32, i32, i32, i32]
        L.iq_prefill_attention.restype = ctypes.c_int
        L.iq_prefill_attention.argtypes = [P, i32, vp, ctypes.c_int, i32, i32, i32, vp, i32, vp, vp, vp, sz, vp]
        L.iq_export_codes.restype = ctypes.c_int
        L.iq_export_codes.argtypes = [P, i32, i32, i32, i32, i32, vp, vp, vp]
        f32, f64, i64 = ctypes.c_float, ctypes.c_double, ctypes.c_int64
        P8, PG, PP = ctypes.POINTER(iq_cache8), ctypes.POINTER(iq_pages), ctypes.POINTER(iq_page_pool)
        for name, res, args in (
            ("iq_cache8_bytes", ctypes.c_int, [i32, i32, i32, i32, ctypes.POINTER(sz)]),
            ("iq_append8", ctypes.c_int, [P8, i32, vp, vp, ctypes.c_int, i64, i64, i32, i32, vp, vp, vp]),
            ("iq_decode8_workspace_size", sz, [i32, i32, i32, i32]),
            ("iq_decode8_attention", ctypes.c_int, [P8, i32, vp, ctypes.c_int, i32, i32, vp, i32, f32, vp, vp, sz, vp]),
            ("iq_prefill8_workspace_size", sz, [i32, i32, i32, i32, i32]),
            ("iq_prefill8_attention", ctypes.c_int, [P8, i32, vp, ctypes.c_int, i32, i32, i32, vp, vp, i32, f32, vp, vp,
                                                     sz, vp]),
            ("iq_export8", ctypes.c_int, [P8, i32, i32, i32, i32, i32, vp, vp]),
            ("iq_rope_frequencies", ctypes.c_int, [i32, f64, i32, f64, f64, f64, f64, vp, ctypes.POINTER(f64)]),
            ("iq_rope", ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, i64, ctypes.c_int, i32, i32, i32, i32, i32, vp, vp,
                                       f32, i32, vp]),
            ("iq_pages_workspace_size", sz, [PG]),
            ("iq_pages_extend", ctypes.c_int, [PG, vp, vp, i32, vp, sz, vp]),
            ("iq_pages_free", ctypes.c_int, [PG, vp, i32, vp]),
            ("iq_pages_fork", ctypes.c_int, [PG, PP, i32, vp, vp, i32, vp, sz, vp]),
            ("iq_pages_compact", ctypes.c_int, [PG, PP, i32, vp, vp, sz, vp]),
            ("iq_pages_copy", ctypes.c_int, [PG, PP, i32, vp, vp, i32, vp, sz, vp]),
        ):
            getattr(L, name).restype = res
            getattr(L, name).argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch

        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, st):
    if st != IQ_OK:
        raise IqError(fn, st)


# ----------------------------------------------------------------------- entry points
def iq_version():
    return lib().iq_version().decode()


def iq_status_string(status):
    return lib().iq_status_string(int(status)).decode()


def iq_cache_bytes(n_layers, n_kv_heads, page_size, n_pages, k_bits=3, v_bits=3):
    a = ctypes.c_size_t(0)
    _check("iq_cache_bytes", lib().iq_cache_bytes(n_layers, n_kv_heads, page_size, n_pages, k_bits, v_bits,
                                                  ctypes.byref(a)))
    return a.value


def iq_init_rotation(seed, n_layers, n_kv_heads):
    """Seeded rotation parameters as a host float32 array [L][Hkv][32][2][4]."""
    out = np.zeros((n_layers, n_kv_heads, 32, 2, 4), dtype=np.float32)
    _check("iq_init_rotation", lib().iq_init_rotation(ctypes.c_uint64(seed), n_layers, n_kv_heads,
                                                      out.ctypes.data_as(ctypes.c_void_p)))
    return out


def iq_rotation_params_per_head(rotation):
    return int(lib().iq_rotation_params_per_head(int(rotation)))


PARAM_SHAPE = {IQ_ROT_ISO: (32, 2, 4), IQ_ROT_QUAT: (32, 4), IQ_ROT_PLANAR: (64, 2)}


def iq_init_rotation_variant(seed, rotation, n_layers, n_kv_heads):
    """Seeded parameters of any rotation variant: host float32 [L][Hkv][...] (see include/iq.h)."""
    rot = ROTATIONS.get(rotation, rotation)
    out = np.zeros((n_layers, n_kv_heads) + PARAM_SHAPE[rot], dtype=np.float32)
    _check("iq_init_rotation_variant", lib().iq_init_rotation_variant(ctypes.c_uint64(seed), rot, n_layers,
                                                                      n_kv_heads, out.ctypes.data_as(ctypes.c_void_p)))
    return out


def iq_encode_append(cache, layer, k, v, start_pos, params, stream=None):
    """k, v: fp16 [batch][n_new][Hkv][128] CUDA tensors (either may be None)."""
    ref = k if k is not None else v
    batch, n_new = int(ref.shape[0]), int(ref.shape[1])
    _check("iq_encode_append", lib().iq_encode_append(ctypes.byref(cache.c), layer, _ptr(k), _ptr(v), batch, n_new,
                                                      _ptr(start_pos), _ptr(params), _stream(stream)))


def iq_decode_workspace_size(batch, n_q_heads, n_kv_heads, max_ctx):
    return int(lib().iq_decode_workspace_size(batch, n_q_heads, n_kv_heads, max_ctx))


def iq_decode_attention(cache, layer, q, ctx_len, max_ctx, params, out, workspace, stream=None):
    """q: [batch][Hq][128] fp16|fp32; out: fp32 [batch][Hq][128]; workspace: uint8 CUDA tensor,
    zero-filled before its first use (torch.zeros); calls leave it ready for the next one."""
    import torch

    dtype = IQ_F32 if q.dtype == torch.float32 else IQ_F16
    _check("iq_decode_attention", lib().iq_decode_attention(
        ctypes.byref(cache.c), layer, _ptr(q), dtype, int(q.shape[0]), int(q.shape[1]), _ptr(ctx_len), int(max_ctx),
        _ptr(params), _ptr(out), _ptr(workspace), int(workspace.numel() * workspace.element_size()), _stream(stream)))


def iq_decode_step(cache, layer, q, k_new, v_new, ctx_len, max_ctx, params, out, workspace, stream=None):
    """Append one token per sequence (k_new, v_new: fp16 [batch][Hkv][128]) at position ctx_len-1 and
    attend over [0, ctx_len)."""
    import torch

    dtype = IQ_F32 if q.dtype == torch.float32 else IQ_F16
    _check("iq_decode_step", lib().iq_decode_step(
        ctypes.byref(cache.c), layer, _ptr(q), dtype, _ptr(k_new), _ptr(v_new), int(q.shape[0]), int(q.shape[1]),
        _ptr(ctx_len), int(max_ctx), _ptr(params), _ptr(out), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream(stream)))


def iq_decode_deferred_workspace_size(batch, n_q_heads, n_kv_heads, max_ctx, max_len):
    return int(lib().iq_decode_deferred_workspace_size(batch, n_q_heads, n_kv_heads, max_ctx, max_len))


def iq_decode_step_deferred(cache, layer, k16, v16, prefix_len, q, k_new, v_new, ctx_len, max_ctx, params, out,
                            workspace, stream=None):
    """Decode step over an fp16 prefix (k16, v16: fp16 [batch][Hkv][max_len][128], prefix_len: int32
    [batch]) followed by the packed cache; the new token is appended (quantised) as by iq_decode_step."""
    import torch

    dtype = IQ_F32 if q.dtype == torch.float32 else IQ_F16
    pre = iq_fp16_prefix(k16.data_ptr(), v16.data_ptr(), prefix_len.data_ptr(), int(k16.shape[2]))
    _check("iq_decode_step_deferred", lib().iq_decode_step_deferred(
        ctypes.byref(cache.c), layer, ctypes.byref(pre), _ptr(q), dtype, _ptr(k_new), _ptr(v_new), int(q.shape[0]),
        int(q.shape[1]), _ptr(ctx_len), int(max_ctx), _ptr(params), _ptr(out), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream(stream)))


def iq_prefill_workspace_size(batch, n_tokens, n_kv_heads, max_ctx):
    return int(lib().iq_prefill_workspace_size(batch, n_tokens, n_kv_heads, max_ctx))


def iq_prefill_attention(cache, layer, q, start_pos, max_ctx, params, out, workspace, stream=None):
    """q: [batch][n_tokens][Hq][128] fp16|fp32; out: fp32 of the same shape; query token i of sequence b
    at position start_pos[b] + i attends causally to the cache's positions 0 .. start_pos[b] + i."""
    import torch

    dtype = IQ_F32 if q.dtype == torch.float32 else IQ_F16
    ws_bytes = 0 if workspace is None else int(workspace.numel() * workspace.element_size())
    _check("iq_prefill_attention", lib().iq_prefill_attention(
        ctypes.byref(cache.c), layer, _ptr(q), dtype, int(q.shape[0]), int(q.shape[1]), int(q.shape[2]),
        _ptr(start_pos), int(max_ctx), _ptr(params), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)))


IQ_NOALLOC_SCRATCH_BYTES = 4 << 20


def iq_decode_attention_noalloc(cache, layer, q, ctx_len, max_ctx, params, out, stream=None):
    """iq_decode_attention with the library's fixed device scratch instead of a caller workspace."""
    import torch

    dtype = IQ_F32 if q.dtype == torch.float32 else IQ_F16
    _check("iq_decode_attention_noalloc", lib().iq_decode_attention_noalloc(
        ctypes.byref(cache.c), layer, _ptr(q), dtype, int(q.shape[0]), int(q.shape[1]), _ptr(ctx_len), int(max_ctx),
        _ptr(params), _ptr(out), _stream(stream)))


def iq_export_codes(cache, layer, kv, seq, t0, n, codes, norms=None, stream=None):
    """codes: uint8 [Hkv][n][128] CUDA tensor; norms: int16/uint16 [Hkv][n] or None."""
    _check("iq_export_codes", lib().iq_export_codes(ctypes.byref(cache.c), layer, kv, seq, t0, n, _ptr(codes),
                                                    _ptr(norms), _stream(stream)))


# ----------------------------------------------------------------------- cache holder
class PagedCache:
    """Device pool of a packed K/V cache (one torch tensor of tile records) and the iq_cache
    struct over it.

    page_size tokens per page (a multiple of 32); with block_table None, sequence b owns page b
    (a contiguous cache of capacity page_size tokens per sequence).  k_bits / v_bits are the
    code widths, rotation the variant ("iso", "quat", "planar" or its IQ_ROT_* value).  The
    k_codes, v_codes, k_norms and v_norms attributes are strided views of the pool's tile records."""

    def __init__(self, n_layers, n_kv_heads, page_size, n_pages, block_table=None, device="cuda", k_bits=3, v_bits=3,
                 rotation=IQ_ROT_ISO):
        import torch

        self.k_bits, self.v_bits = k_bits, v_bits
        self.rotation = ROTATIONS.get(rotation, rotation)
        self.tile_bytes = tile_bytes(k_bits, v_bits)
        self.pool = torch.empty(iq_cache_bytes(n_layers, n_kv_heads, page_size, n_pages, k_bits, v_bits),
                                dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.block_table = block_table
        self.n_layers, self.n_kv_heads, self.page_size, self.n_pages = n_layers, n_kv_heads, page_size, n_pages
        self.max_pages_per_seq = int(block_table.shape[1]) if block_table is not None else 1
        t = self.tiles()
        kv0 = 32 * k_record_bytes(k_bits)
        kn0 = kv0 + 2 * v_block_bytes(v_bits)
        self.k_codes = t[..., 0:kv0]
        self.v_codes = t[..., kv0:kn0]
        self.k_norms = t[..., kn0:kn0 + 64].view(torch.int16)
        self.v_norms = t[..., kn0 + 64:kn0 + 128].view(torch.int16)
        self.c = iq_cache(
            self.pool.data_ptr(), n_layers, n_kv_heads, HEAD_DIM, page_size, n_pages,
            block_table.data_ptr() if block_table is not None else None,
            self.max_pages_per_seq, self.status.data_ptr(), k_bits, v_bits, self.rotation,
        )

    def tiles(self):
        """[L][n_pages][Hkv][page_size/32][tile_bytes] tile records."""
        return self.pool.view(self.n_layers, self.n_pages, self.n_kv_heads, self.page_size // TILE_TOKENS,
                              self.tile_bytes)

    # Views with the records' logical shapes (for writing oracle-made records in tests).
    def k_code_view(self):
        """[L][n_pages][Hkv][page_size/32][32][16 k_bits]"""
        return self.k_codes.view(*self.k_codes.shape[:-1], TILE_TOKENS, k_record_bytes(self.k_bits))

    def v_code_view(self):
        """[L][n_pages][Hkv][page_size/32][2][256 v_bits]"""
        return self.v_codes.view(*self.v_codes.shape[:-1], 2, v_block_bytes(self.v_bits))

    def k_norm_view(self):
        """[L][n_pages][Hkv][page_size/32][32] int16"""
        return self.k_norms

    def v_norm_view(self):
        return self.v_norms


# ----------------------------------------------------------------------- the 8-bit cache, rotary positions, pages
# These calls run on the device of their tensors, whichever is current, and on that device's current
# stream unless one is given.  A tensor of the wrong shape, type, layout or device is a ValueError.
def _bad(fn, what):
    raise ValueError(f"{fn}: {what}")


_dtypes = {}  # torch's number types -> the library's; and "i32", "f64"


def _types():
    if not _dtypes:
        import torch

        _dtypes.update({torch.float16: IQ_F16, torch.bfloat16: IQ_BF16, torch.float32: IQ_F32, "i32": torch.int32,
                        "f64": torch.float64, "torch": torch})
    return _dtypes


def _dtype(fn, t):
    d = _types().get(t.dtype)
    if d is None:
        _bad(fn, f"float16, bfloat16 or float32 wanted, got {t.dtype}")
    return d


def _plain(fn, name, t, dev, dtype, shape):
    """The address of a contiguous tensor of this type, shape and device."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _bad(fn, f"{name}: a contiguous {dtype} tensor of shape {shape} on cuda:{dev} wanted, got {t.dtype} "
                 f"{tuple(t.shape)}, strides {t.stride()}, on {t.device}")
    return t.data_ptr()


def _i32(fn, name, t, dev, n):
    return _plain(fn, name, t, dev, _types()["i32"], (n,))


def _bytes(fn, name, t, dev):
    """(address, bytes) of a workspace."""
    if t.get_device() != dev or not t.is_contiguous():
        _bad(fn, f"{name}: a contiguous tensor on cuda:{dev} wanted")
    return t.data_ptr(), t.numel() * t.element_size()


_fns = {}  # the library's functions by name


def _run8(fn, dev, stream, *args):
    """The C call `fn` on device `dev`, its stream last."""
    torch = _types()["torch"]
    if dev < 0:
        _bad(fn, "CUDA tensors wanted")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)  # (a tenth of current_stream()'s time)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    f = _fns.get(fn)
    if f is None or _lib is None:
        f = _fns[fn] = getattr(lib(), fn)
    if torch.cuda.current_device() == dev:
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st != IQ_OK:
        raise IqError(fn, st)


def iq_cache8_bytes(n_layers, n_kv_heads, page_size, n_pages):
    a = ctypes.c_size_t(0)
    _check("iq_cache8_bytes", lib().iq_cache8_bytes(n_layers, n_kv_heads, page_size, n_pages, ctypes.byref(a)))
    return a.value


class PagedCache8:
    """Device pool of an 8-bit K/V cache (one torch tensor of tile records) and the iq_cache8 struct over
    it.  page_size, n_pages and block_table as for PagedCache; code "e4m3" or "s8" (or its IQ_* value);
    pool: the uint8 tensor to use instead of a new one."""

    def __init__(self, n_layers, n_kv_heads, page_size, n_pages, block_table=None, device="cuda", code="e4m3", pool=None):
        import torch

        need = iq_cache8_bytes(n_layers, n_kv_heads, page_size, n_pages)
        if pool is None:
            pool = torch.empty(need, dtype=torch.uint8, device=device)
        self.dev = pool.get_device()
        _plain("PagedCache8", "pool", pool, self.dev, torch.uint8, (need,))
        self.pool, self.block_table = pool, block_table
        self.code = CODES8.get(code, code)
        self.status = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self.n_layers, self.n_kv_heads, self.page_size, self.n_pages = n_layers, n_kv_heads, page_size, n_pages
        self.max_pages_per_seq = 1
        table = None
        if block_table is not None:
            if block_table.dim() != 2:
                _bad("PagedCache8", "block_table: [batch][max_pages_per_seq] wanted")
            self.max_pages_per_seq = int(block_table.shape[1])
            table = _plain("PagedCache8", "block_table", block_table, self.dev, torch.int32, tuple(block_table.shape))
        self.max_batch = n_pages if block_table is None else int(block_table.shape[0])
        self.c = iq_cache8(pool.data_ptr(), n_layers, n_kv_heads, HEAD_DIM, page_size, n_pages, table,
                           self.max_pages_per_seq, self.status.data_ptr(), self.code)
        self.ref = ctypes.byref(self.c)

    def tiles(self):
        """[L][n_pages][Hkv][page_size/32][8224] tile records."""
        return self.pool.view(self.n_layers, self.n_pages, self.n_kv_heads, self.page_size // TILE_TOKENS, TILE8_BYTES)


def _batch8(fn, cache, batch):
    if batch > cache.max_batch:
        _bad(fn, f"{batch} sequences, and rows for {cache.max_batch} in the cache")


def iq_append8(cache, layer, k, v, start_pos, n_valid=None, stream=None):
    """k, v: fp16, bf16 or fp32 [batch][n_new][Hkv][128] CUDA tensors (either may be None), whose heads are
    contiguous and whose tokens are equally far apart (slices of a fused projection's rows are); start_pos,
    n_valid: int32 [batch]."""
    fn, dev = "iq_append8", cache.dev
    x = k if k is not None else v
    if x is None:
        _bad(fn, "k or v wanted")
    if x.dim() != 4:
        _bad(fn, "[batch][n_new][Hkv][128] tensors wanted")
    batch, n = x.shape[0], x.shape[1]
    _batch8(fn, cache, batch)
    if batch == 0 or n == 0:
        return
    strides, shape = [], (batch, n, cache.n_kv_heads, HEAD_DIM)
    for t in (k, v):
        if t is None:
            strides.append(0)
            continue
        ok, stride = t.dtype == x.dtype and t.get_device() == dev and t.shape == shape, 0  # 0: contiguous rows
        if ok and not t.is_contiguous():
            st = t.stride()
            stride = st[1] if n > 1 else st[0] if batch > 1 else 0
            ok = (st[3] == 1 and (shape[2] == 1 or st[2] == HEAD_DIM) and (batch == 1 or st[0] == n * stride)
                  and (batch * n == 1 or stride >= shape[2] * HEAD_DIM))  # (a broadcast tensor's is 0)
        if not ok:
            _bad(fn, f"[{batch}][{n}][{cache.n_kv_heads}][128] tensors of one type, with contiguous heads and equally "
                     f"distant tokens, on cuda:{dev} wanted, got {t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device}")
        strides.append(stride)
    _run8(fn, dev, stream, cache.ref, layer, k.data_ptr() if k is not None else None,
          v.data_ptr() if v is not None else None, _dtype(fn, x), *strides, batch, n,
          _i32(fn, "start_pos", start_pos, dev, batch),
          None if n_valid is None else _i32(fn, "n_valid", n_valid, dev, batch))


def iq_decode8_workspace_size(batch, n_q_heads, n_kv_heads, max_ctx):
    return int(lib().iq_decode8_workspace_size(batch, n_q_heads, n_kv_heads, max_ctx))


def iq_decode8_attention(cache, layer, q, ctx_len, max_ctx, out, workspace, scale=None, stream=None):
    """q, out: [batch][Hq][128], fp16, bf16 or fp32; ctx_len: int32 [batch]; workspace: zero-filled before its
    first use, as iq_decode_attention's; scale: of the scores, 1/sqrt(128) by default."""
    fn, dev = "iq_decode8_attention", cache.dev
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        _bad(fn, "q: [batch][Hq][128] wanted")
    shape = tuple(q.shape)
    _batch8(fn, cache, shape[0])
    if q.numel() == 0:
        return
    ws, nbytes = _bytes(fn, "workspace", workspace, dev)
    _run8(fn, dev, stream, cache.ref, layer, _plain(fn, "q", q, dev, q.dtype, shape), _dtype(fn, q), shape[0], shape[1],
          _i32(fn, "ctx_len", ctx_len, dev, shape[0]), max_ctx, HEAD_DIM ** -0.5 if scale is None else scale,
          _plain(fn, "out", out, dev, q.dtype, shape), ws, nbytes)


def iq_prefill8_workspace_size(batch, n_tokens, n_q_heads, n_kv_heads, max_ctx):
    return int(lib().iq_prefill8_workspace_size(batch, n_tokens, n_q_heads, n_kv_heads, max_ctx))


def iq_prefill8_attention(cache, layer, q, start_pos, max_ctx, out, workspace, n_valid=None, scale=None, stream=None):
    """q, out: [batch][n_tokens][Hq][128], fp16, bf16 or fp32; query token i of sequence b at position start_pos[b]
    + i attends causally; n_valid: int32 [batch], the tokens that are there (rows of out behind them stay as they
    were)."""
    fn, dev = "iq_prefill8_attention", cache.dev
    if q.dim() != 4 or q.shape[3] != HEAD_DIM:
        _bad(fn, "q: [batch][n_tokens][Hq][128] wanted")
    shape = tuple(q.shape)
    _batch8(fn, cache, shape[0])
    if q.numel() == 0:
        return
    ws, nbytes = _bytes(fn, "workspace", workspace, dev)
    _run8(fn, dev, stream, cache.ref, layer, _plain(fn, "q", q, dev, q.dtype, shape), _dtype(fn, q), shape[0], shape[1],
          shape[2], _i32(fn, "start_pos", start_pos, dev, shape[0]),
          None if n_valid is None else _i32(fn, "n_valid", n_valid, dev, shape[0]), max_ctx,
          HEAD_DIM ** -0.5 if scale is None else scale, _plain(fn, "out", out, dev, q.dtype, shape), ws, nbytes)


def iq_export8(cache, layer, kv, seq, t0, n, values, stream=None):
    """values: float32 [Hkv][n][128] CUDA tensor."""
    import torch

    fn = "iq_export8"
    if seq >= cache.max_batch:
        _bad(fn, f"sequence {seq}, and rows for {cache.max_batch} in the cache")
    if n == 0:
        return
    _run8(fn, cache.dev, stream, cache.ref, layer, kv, seq, t0, n,
          _plain(fn, "values", values, cache.dev, torch.float32, (cache.n_kv_heads, n, HEAD_DIM)))


def iq_rope_frequencies(rotary_dim, base=10000.0, scaling="plain", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """(float64 [rotary_dim/2] radians per position, factor on q and k); scalings as in include/iq8.h."""
    out, ms = np.zeros(max(0, rotary_dim // 2), dtype=np.float64), ctypes.c_double(0.0)
    _check("iq_rope_frequencies", lib().iq_rope_frequencies(
        rotary_dim, base, ROPE_SCALINGS.get(scaling, scaling), factor, original_len, low, high,
        out.ctypes.data_as(ctypes.c_void_p), ctypes.byref(ms)))
    return out, ms.value


def _rope_side(fn, name, x, y, dtype, dev, n):
    """(address, row stride, out address, out row stride, heads) of q or k."""
    if x is None or y is None:
        if x is not None or y is not None:
            _bad(fn, f"{name} and {name}_out belong together")
        return None, 0, None, 0, 0
    heads = x.shape[1] if x.dim() == 3 else 0
    shape, strides = (n, heads, HEAD_DIM), []
    for t in (x,) if y is x else (x, y):
        ok, stride = t.dtype == dtype and t.get_device() == dev and t.shape == shape, 0  # 0: contiguous rows
        if ok and not t.is_contiguous():
            st = t.stride()
            stride = st[0] if n > 1 else 0
            ok = st[2] == 1 and (heads == 1 or st[1] == HEAD_DIM) and (n == 1 or stride >= heads * HEAD_DIM)  # (broadcast: 0)
        if not ok:
            _bad(fn, f"{name}: [{n}][heads][128] tensors of one type with contiguous heads on cuda:{dev} wanted, got "
                     f"{t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device}")
        strides.append(stride)
    return x.data_ptr(), strides[0], y.data_ptr(), strides[-1], heads


def iq_rope(q, k, positions, freq, q_out=None, k_out=None, layout="half", mscale=1.0, inverse=False, stream=None):
    """q, k: fp16, bf16 or fp32 [n_tokens][heads][128] (either may be None), rows as far apart as they may be;
    q_out, k_out: where the results go, by default q and k themselves; positions: int32 [n_tokens]; freq:
    float64 [rotary_dim/2] (iq_rope_frequencies)."""
    fn = "iq_rope"
    x = q if q is not None else k
    if x is None:
        _bad(fn, "q or k wanted")
    if x.dim() != 3:
        _bad(fn, "[n_tokens][heads][128] tensors wanted")
    dev, n, pairs = x.get_device(), x.shape[0], freq.numel()
    if n == 0:
        return
    a = _rope_side(fn, "q", q, q if q_out is None else q_out, x.dtype, dev, n)
    b = _rope_side(fn, "k", k, k if k_out is None else k_out, x.dtype, dev, n)
    _run8(fn, dev, stream, *a[:4], *b[:4], _dtype(fn, x), n, a[4], b[4], 2 * pairs, ROPE_LAYOUTS.get(layout, layout),
          _i32(fn, "positions", positions, dev, n), _plain(fn, "freq", freq, dev, _types()["f64"], (pairs,)), mscale,
          1 if inverse else 0)


class PageTable:
    """Block table, lengths and page counts of up to max_seqs sequences (give .block_table to the caches), and
    the workspace of the operations on them.  Tensors given are used as they are."""

    def __init__(self, max_seqs, max_pages_per_seq, page_size, n_pages, device="cuda", block_table=None, seq_len=None,
                 ref=None):
        import torch

        if block_table is None:
            block_table = torch.full((max_seqs, max_pages_per_seq), -1, dtype=torch.int32, device=device)
        device = block_table.device
        if seq_len is None:
            seq_len = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        if ref is None:
            ref = torch.zeros(n_pages, dtype=torch.int32, device=device)
        self.dev = block_table.get_device()
        self.block_table, self.seq_len, self.ref = block_table, seq_len, ref
        self.page_size, self.n_pages = page_size, n_pages
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.c = iq_pages(
            _plain("PageTable", "block_table", block_table, self.dev, torch.int32, (max_seqs, max_pages_per_seq)),
            _i32("PageTable", "seq_len", seq_len, self.dev, max_seqs), _i32("PageTable", "ref", ref, self.dev, n_pages),
            max_seqs, max_pages_per_seq, page_size, n_pages, self.status.data_ptr())
        self.p = ctypes.byref(self.c)
        need = int(lib().iq_pages_workspace_size(self.p))
        if not need:
            _bad("PageTable", "sizes of at least 1 and a page_size that is a multiple of 32 wanted")
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)
        self.ws = self.workspace.data_ptr(), need


class PagePool:
    """The pool of a cache (or several: PagePool.of(cache, ...)) whose pages a PageTable's operations move."""

    def __init__(self, pool, n_layers, n_kv_heads, page_size, n_pages, tile_bytes):
        import torch

        self.page_size, self.n_pages, self.n, self.dev = page_size, n_pages, 1, pool.get_device()
        self.held = [pool]
        need = n_layers * n_pages * n_kv_heads * (page_size // TILE_TOKENS) * tile_bytes
        addr = _plain("PagePool", "pool", pool, self.dev, torch.uint8, (need,))
        self.c = (iq_page_pool * 1)(iq_page_pool(addr, n_layers, n_kv_heads, tile_bytes))

    @classmethod
    def of(cls, *caches):
        """The pools of caches of either kind that share a block table."""
        if not caches:
            _bad("PagePool", "a cache wanted")
        each = [cls(c.pool, c.n_layers, c.n_kv_heads, c.page_size, c.n_pages, getattr(c, "tile_bytes", TILE8_BYTES))
                for c in caches]
        one = each[0]
        if any((e.page_size, e.n_pages, e.dev) != (one.page_size, one.n_pages, one.dev) for e in each):
            _bad("PagePool", "caches of one page size, number of pages and device wanted")
        one.n, one.held = len(each), [e.held[0] for e in each]
        one.c = (iq_page_pool * len(each))(*(e.c[0] for e in each))
        return one


def _pools(fn, table, pools):
    if pools is None:
        return None, 0
    if (pools.page_size, pools.n_pages, pools.dev) != (table.page_size, table.n_pages, table.dev):
        _bad(fn, "the pools' page size, number of pages and device are not the table's")
    return pools.c, pools.n


def iq_pages_extend(table, ids, new_len, stream=None):
    """Sequences ids grow to new_len tokens (int32 [n] each) and get their pages."""
    fn, n = "iq_pages_extend", ids.numel()
    _run8(fn, table.dev, stream, table.p, _i32(fn, "ids", ids, table.dev, n), _i32(fn, "new_len", new_len, table.dev, n), n,
          *table.ws)


def iq_pages_free(table, ids, stream=None):
    fn, n = "iq_pages_free", ids.numel()
    _run8(fn, table.dev, stream, table.p, _i32(fn, "ids", ids, table.dev, n), n)


def iq_pages_fork(table, pools, parent, child, stream=None):
    """Empty sequences child become copies of parent (int32 [n] each); pools: a PagePool, or None."""
    fn, n = "iq_pages_fork", parent.numel()
    c, m = _pools(fn, table, pools)
    _run8(fn, table.dev, stream, table.p, c, m, _i32(fn, "parent", parent, table.dev, n),
          _i32(fn, "child", child, table.dev, n), n, *table.ws)


def iq_pages_compact(table, pools, n_held=None, stream=None):
    """The held pages move to the front; n_held: int32 [1] that gets their number, or None."""
    fn = "iq_pages_compact"
    c, m = _pools(fn, table, pools)
    _run8(fn, table.dev, stream, table.p, c, m, None if n_held is None else _i32(fn, "n_held", n_held, table.dev, 1),
          *table.ws)


def iq_pages_copy(table, pools, src, dst, stream=None):
    """Page src[i] of every layer to page dst[i] (int32 [n] each)."""
    fn, n = "iq_pages_copy", src.numel()
    c, m = _pools(fn, table, pools)
    _run8(fn, table.dev, stream, table.p, c, m, _i32(fn, "src", src, table.dev, n), _i32(fn, "dst", dst, table.dev, n), n,
          *table.ws)
