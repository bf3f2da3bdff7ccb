"""Python binding of libfa (exact attention for GB300 / sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libfa.so.  The C functions keep their names (`fa_fwd`, `fa_bwd`,
...); each takes device pointers (ints or torch CUDA tensors) and raises
`FaError` on a non-OK status.  `forward` / `backward` are conveniences that
allocate the outputs with torch and call the same C functions; they accept
[B, H, N, d] views of any layout whose last dimension is contiguous (for
example a [B, N, H, d] buffer transposed to [B, H, N, d]) and pass each
tensor's strides to the *_ex calls, so nothing is copied; they also take
dropout (probability, seed, offset).

Importing this package fails loudly if libfa.so has not been built
(`python -c "import __graft_entry__ as g; g.build()"`): there is no fallback.
"""
import contextlib
import ctypes
import os

__all__ = [
    "FaError", "FaMask", "FaLayout", "FaLayouts", "FaDropout", "FaBias", "FaOptions", "layout_of",
    "bias_of",
    "make_layouts", "make_options", "fa_fwd_ex", "fa_bwd_ex", "fa_fwd_fp32_ex", "fa_bwd_fp32_ex",
    "fa_bwd_preprocess_ex", "fa_bwd_dkdv_ex", "fa_bwd_dq_ex",
    "lib", "fa_fwd", "fa_bwd", "fa_bwd_workspace_size",
    "fa_bwd_preprocess", "fa_bwd_dkdv", "fa_bwd_dq", "fa_fwd_fp32", "fa_bwd_fp32",
    "fa_bwd_noalloc", "NOALLOC_SCRATCH_BYTES", "fa_status_string", "fa_get_device_status", "fa_debug_wait_timeout",
    "make_mask", "forward", "backward", "LIB_PATH",
    "fa_block_mask_order", "fa_block_mask_order_len", "block_mask_order",
    "FaRotary", "FaRopeLayouts", "FaCache", "FaCacheLayouts", "FA_CACHE_BF16", "FA_CACHE_E4M3",
    "fa_rope", "fa_rope_bwd", "fa_rope_fp32", "fa_rope_bwd_fp32", "fa_cache_write",
    "fa_cache_read", "fa_cache_fwd", "fa_cache_fwd_workspace_size",
    "Rope", "rope_frequencies", "rope", "rope_backward", "KVCache", "cache_write", "cache_read",
    "cache_forward", "decode_step", "tree_mask",
    "FA_MASK_NONE", "FA_MASK_KEY_PADDING", "FA_MASK_BLOCK_SPARSE", "STATUS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

FA_MASK_NONE, FA_MASK_KEY_PADDING, FA_MASK_BLOCK_SPARSE = 0, 1, 2
FA_CACHE_BF16, FA_CACHE_E4M3 = 0, 1
STATUS = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_ALIGNMENT",
          4: "FA_ERR_WORKSPACE", 5: "FA_ERR_CUDA", 6: "FA_ERR_TIMEOUT", 7: "FA_ERR_PAGE"}


class FaError(RuntimeError):
    def __init__(self, code, where, detail=None):
        self.code = code
        msg = "%s returned %s" % (where, STATUS.get(code, code))
        if detail:
            msg += " (%s)" % detail
        super().__init__(msg)


class FaMask(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("kv_len", ctypes.c_void_p),
                ("block_mask", ctypes.c_void_p), ("block_size", ctypes.c_int),
                ("tile_order", ctypes.c_void_p)]


class FaLayout(ctypes.Structure):
    """Element strides of one [B, H, N, d] tensor (fa_layout)."""
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("row", ctypes.c_int64)]


_LAYOUT_NAMES = ("q", "k", "v", "o", "dO", "dq", "dk", "dv")


class FaLayouts(ctypes.Structure):
    """Layouts of the tensors of one call (fa_layouts)."""
    _fields_ = [(n, FaLayout) for n in _LAYOUT_NAMES]


class FaDropout(ctypes.Structure):
    """Dropout of a call (fa_dropout): probability, generator seed, offset."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint32)]


class FaBias(ctypes.Structure):
    """Additive score bias (fa_bias): fp32 device pointer and element strides."""
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", ctypes.c_int64), ("head", ctypes.c_int64),
                ("row", ctypes.c_int64)]


class FaOptions(ctypes.Structure):
    """Options of the *_ex calls (fa_options)."""
    _fields_ = [("layouts", ctypes.POINTER(FaLayouts)), ("dropout", ctypes.POINTER(FaDropout)),
                ("bias", ctypes.POINTER(FaBias))]


class FaRotary(ctypes.Structure):
    """Rotary positions of a call (fa_rotary)."""
    _fields_ = [("freq", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("pos_stride", ctypes.c_int64), ("dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("factor", ctypes.c_float)]


class FaRopeLayouts(ctypes.Structure):
    """Layouts of the tensors of a rotation (fa_rope_layouts)."""
    _fields_ = [(n, FaLayout) for n in ("q", "k", "q_out", "k_out")]


class FaCache(ctypes.Structure):
    """A paged key/value cache (fa_cache)."""
    _fields_ = [("format", ctypes.c_int), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("d", ctypes.c_int), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("layout", ctypes.POINTER(FaLayout)),
                ("scale_layout", ctypes.POINTER(FaLayout)), ("block_table", ctypes.c_void_p),
                ("table_width", ctypes.c_int), ("table_stride", ctypes.c_int64)]


class FaCacheLayouts(ctypes.Structure):
    """Layouts of the dense k and v of a cache call (fa_cache_layouts)."""
    _fields_ = [("k", FaLayout), ("v", FaLayout)]


if not os.path.exists(LIB_PATH):
    raise ImportError("libfa.so is not built (expected at %s); run "
                      "__graft_entry__.build() first" % LIB_PATH)
lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_mp = ctypes.POINTER(FaMask)
_op = ctypes.POINTER(FaOptions)
_lp = ctypes.POINTER(FaLayout)
_rp = ctypes.POINTER(FaRotary)
_rlp = ctypes.POINTER(FaRopeLayouts)
_cp = ctypes.POINTER(FaCache)
_clp = ctypes.POINTER(FaCacheLayouts)

_SIGS = {
    "fa_fwd": [_p, _p, _p, _p, _p, _i, _i, _i, _i, _f, _i, _mp, _p],
    "fa_fwd_fp32": [_p, _p, _p, _p, _p, _i, _i, _i, _i, _f, _i, _mp, _p],
    "fa_bwd_workspace_size": [_i, _i, _i, _i],
    "fa_bwd": [_p] * 10 + [_sz, _i, _i, _i, _i, _f, _i, _mp, _p],
    "fa_bwd_fp32": [_p] * 10 + [_sz, _i, _i, _i, _i, _f, _i, _mp, _p],
    "fa_bwd_preprocess": [_p, _p, _p, _i, _i, _i, _i, _p],
    "fa_bwd_dkdv": [_p] * 8 + [_i, _i, _i, _i, _f, _i, _mp, _p],
    "fa_bwd_dq": [_p] * 7 + [_i, _i, _i, _i, _f, _i, _mp, _p],
    "fa_status_string": [_i],
    "fa_get_device_status": [_p, ctypes.POINTER(ctypes.c_int)],
    "fa_debug_wait_timeout": [ctypes.c_uint, _p],
    "fa_bwd_noalloc": [_p] * 9 + [_i, _i, _i, _i, _f, _i, _mp, _p],
    "fa_last_cuda_error": [],
    "fa_fwd_ex": [_p, _p, _p, _p, _p, _i, _i, _i, _i, _f, _i, _mp, _op, _p],
    "fa_fwd_fp32_ex": [_p, _p, _p, _p, _p, _i, _i, _i, _i, _f, _i, _mp, _op, _p],
    "fa_bwd_ex": [_p] * 10 + [_sz, _i, _i, _i, _i, _f, _i, _mp, _op, _p],
    "fa_bwd_fp32_ex": [_p] * 10 + [_sz, _i, _i, _i, _i, _f, _i, _mp, _op, _p],
    "fa_bwd_preprocess_ex": [_p, _p, _p, _i, _i, _i, _i, _op, _p],
    "fa_bwd_dkdv_ex": [_p] * 8 + [_i, _i, _i, _i, _f, _i, _mp, _op, _p],
    "fa_bwd_dq_ex": [_p] * 7 + [_i, _i, _i, _i, _f, _i, _mp, _op, _p],
    "fa_rope": [_p] * 4 + [_i] * 5 + [_rp, _rlp, _p],
    "fa_rope_bwd": [_p] * 4 + [_i] * 5 + [_rp, _rlp, _p],
    "fa_rope_fp32": [_p] * 4 + [_i] * 5 + [_rp, _rlp, _p],
    "fa_rope_bwd_fp32": [_p] * 4 + [_i] * 5 + [_rp, _rlp, _p],
    "fa_cache_write": [_p, _p, _cp, _p, _p, _i, _i, _rp, _clp, _p],
    "fa_cache_read": [_cp, _p, _p, _p, _p, _i, _i, _clp, _p],
    "fa_cache_fwd_workspace_size": [_i] * 5,
    "fa_cache_fwd": [_p, _cp] + [_p] * 6 + [_sz, _i, _i, _i, _f, _lp, _lp, _p],
    "fa_block_mask_order_len": [_i],
    "fa_block_mask_order": [_p, _i, _i, _p, _p],
}
for _name, _args in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int
lib.fa_bwd_workspace_size.restype = ctypes.c_size_t
lib.fa_cache_fwd_workspace_size.restype = ctypes.c_size_t
lib.fa_status_string.restype = ctypes.c_char_p
lib.fa_last_cuda_error.restype = ctypes.c_char_p


def _ptr(x):
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _stream(s):
    if s is None:
        return None
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


def _check(code, where):
    if code != 0:
        detail = lib.fa_last_cuda_error().decode() if code == 5 else None
        raise FaError(code, where, detail)


def make_mask(kv_len=None, block_mask=None, block_size=128, tile_order=None):
    """A pointer to an fa_mask for key padding (kv_len) or a block-sparse tile
    mask (device tensors), or None for no mask.  tile_order: the block mask's
    work order (block_mask_order), or None for the default order."""
    if kv_len is not None and block_mask is not None:
        raise ValueError("one mask kind at a time")
    if tile_order is not None and block_mask is None:
        raise ValueError("tile_order belongs to a block mask")
    if kv_len is not None:
        return ctypes.pointer(FaMask(FA_MASK_KEY_PADDING, _ptr(kv_len), None, block_size, None))
    if block_mask is not None:
        return ctypes.pointer(FaMask(FA_MASK_BLOCK_SPARSE, None, _ptr(block_mask), block_size,
                                     _ptr(tile_order)))
    return None


def layout_of(t):
    """FaLayout of a 4-D [B, H, N, d] tensor whose last dimension is contiguous."""
    if t.dim() != 4:
        raise ValueError("expected a [B, H, N, d] tensor")
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError("the d elements of a row must be contiguous (stride(3) == 1)")
    return FaLayout(t.stride(0), t.stride(1), t.stride(2))


def make_layouts(**tensors):
    """An FaLayouts holding layout_of(t) for each named tensor (names: q, k,
    v, o, dO, dq, dk, dv); entries not given stay zero, which the calls that
    read them reject."""
    unknown = set(tensors) - set(_LAYOUT_NAMES)
    if unknown:
        raise ValueError("unknown tensor names: %s" % sorted(unknown))
    ls = FaLayouts()
    for name, t in tensors.items():
        setattr(ls, name, layout_of(t))
    return ls


def bias_of(t):
    """FaBias of a CUDA fp32 tensor broadcastable to [B, H, N, N] (4-D, last
    dimension contiguous); dimensions of size 1 are broadcast (stride 0)."""
    if t.dim() != 4:
        raise ValueError("the bias must be 4-D: [B or 1, H or 1, N, N]")
    if t.stride(3) != 1:
        raise ValueError("the bias columns must be contiguous")
    st = [0 if t.shape[i] == 1 else t.stride(i) for i in range(3)]
    return FaBias(t.data_ptr(), st[0], st[1], st[2])


def make_options(layouts=None, dropout_p=0.0, seed=0, offset=0, bias=None):
    """A pointer to an FaOptions: `layouts` an FaLayouts (or None: dense),
    dropout with probability dropout_p (0: none), generator seed and offset,
    `bias` an FaBias (or None).  The pointer keeps its members alive."""
    opt = FaOptions()
    keep = []
    if bias is not None:
        keep.append(bias)
        opt.bias = ctypes.pointer(bias)
    if layouts is not None:
        keep.append(layouts)
        opt.layouts = ctypes.pointer(layouts)
    if dropout_p:
        dr = FaDropout(dropout_p, seed, offset)
        keep.append(dr)
        opt.dropout = ctypes.pointer(dr)
    ptr = ctypes.pointer(opt)
    ptr._keep = keep
    return ptr


def fa_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, mask=None, options=None,
              stream=None):
    _check(lib.fa_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, scale,
                         int(causal), mask, options, _stream(stream)), "fa_fwd_ex")


def fa_fwd_fp32_ex(q, k, v, o, lse, B, H, N, d, scale, causal, mask=None, options=None,
                   stream=None):
    _check(lib.fa_fwd_fp32_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, scale,
                              int(causal), mask, options, _stream(stream)), "fa_fwd_fp32_ex")


def fa_bwd_ex(q, k, v, o, dO, lse, dq, dk, dv, workspace, workspace_bytes, B, H, N, d, scale,
              causal, mask=None, options=None, stream=None):
    _check(lib.fa_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                         _ptr(dk), _ptr(dv), _ptr(workspace), workspace_bytes, B, H, N, d, scale,
                         int(causal), mask, options, _stream(stream)), "fa_bwd_ex")


def fa_bwd_fp32_ex(q, k, v, o, dO, lse, dq, dk, dv, workspace, workspace_bytes, B, H, N, d,
                   scale, causal, mask=None, options=None, stream=None):
    _check(lib.fa_bwd_fp32_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                              _ptr(dk), _ptr(dv), _ptr(workspace), workspace_bytes, B, H, N, d,
                              scale, int(causal), mask, options, _stream(stream)),
           "fa_bwd_fp32_ex")


def fa_bwd_preprocess_ex(o, dO, D, B, H, N, d, options=None, stream=None):
    _check(lib.fa_bwd_preprocess_ex(_ptr(o), _ptr(dO), _ptr(D), B, H, N, d, options,
                                    _stream(stream)), "fa_bwd_preprocess_ex")


def fa_bwd_dkdv_ex(q, k, v, dO, lse, D, dk, dv, B, H, N, d, scale, causal, mask=None,
                   options=None, stream=None):
    _check(lib.fa_bwd_dkdv_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(D), _ptr(dk),
                              _ptr(dv), B, H, N, d, scale, int(causal), mask, options,
                              _stream(stream)), "fa_bwd_dkdv_ex")


def fa_bwd_dq_ex(q, k, v, dO, lse, D, dq, B, H, N, d, scale, causal, mask=None, options=None,
                 stream=None):
    _check(lib.fa_bwd_dq_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(D), _ptr(dq),
                            B, H, N, d, scale, int(causal), mask, options, _stream(stream)),
           "fa_bwd_dq_ex")


def fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, mask=None, stream=None):
    _check(lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, scale,
                      int(causal), mask, _stream(stream)), "fa_fwd")


def fa_fwd_fp32(q, k, v, o, lse, B, H, N, d, scale, causal, mask=None, stream=None):
    _check(lib.fa_fwd_fp32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, scale,
                           int(causal), mask, _stream(stream)), "fa_fwd_fp32")


def fa_bwd_workspace_size(B, H, N, d):
    return lib.fa_bwd_workspace_size(B, H, N, d)


def fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, workspace, workspace_bytes, B, H, N, d, scale,
           causal, mask=None, stream=None):
    _check(lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                      _ptr(dk), _ptr(dv), _ptr(workspace), workspace_bytes, B, H, N, d, scale,
                      int(causal), mask, _stream(stream)), "fa_bwd")


def fa_bwd_fp32(q, k, v, o, dO, lse, dq, dk, dv, workspace, workspace_bytes, B, H, N, d, scale,
                causal, mask=None, stream=None):
    _check(lib.fa_bwd_fp32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                           _ptr(dk), _ptr(dv), _ptr(workspace), workspace_bytes, B, H, N, d,
                           scale, int(causal), mask, _stream(stream)), "fa_bwd_fp32")


def fa_bwd_preprocess(o, dO, D, B, H, N, d, stream=None):
    _check(lib.fa_bwd_preprocess(_ptr(o), _ptr(dO), _ptr(D), B, H, N, d, _stream(stream)),
           "fa_bwd_preprocess")


def fa_bwd_dkdv(q, k, v, dO, lse, D, dk, dv, B, H, N, d, scale, causal, mask=None, stream=None):
    _check(lib.fa_bwd_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(D), _ptr(dk),
                           _ptr(dv), B, H, N, d, scale, int(causal), mask, _stream(stream)),
           "fa_bwd_dkdv")


def fa_bwd_dq(q, k, v, dO, lse, D, dq, B, H, N, d, scale, causal, mask=None, stream=None):
    _check(lib.fa_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(D), _ptr(dq),
                         B, H, N, d, scale, int(causal), mask, _stream(stream)), "fa_bwd_dq")


NOALLOC_SCRATCH_BYTES = 32 << 20   # FA_NOALLOC_SCRATCH_BYTES


def fa_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, mask=None,
                   stream=None):
    """fa_bwd without a workspace argument, for callers that cannot allocate
    device memory: the library's fixed scratch array is used instead (sizes
    whose workspace exceeds NOALLOC_SCRATCH_BYTES raise FaError)."""
    _check(lib.fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, H, N, d, scale, int(causal), mask,
                              _stream(stream)), "fa_bwd_noalloc")


def fa_block_mask_order_len(T):
    return lib.fa_block_mask_order_len(T)


def fa_block_mask_order(block_mask, T, causal, tile_order, stream=None):
    _check(lib.fa_block_mask_order(_ptr(block_mask), T, int(causal), _ptr(tile_order),
                                   _stream(stream)), "fa_block_mask_order")


def block_mask_order(block_mask, causal=False, stream=None):
    """The work order of a [T, T] uint8 CUDA block mask (an int32 CUDA
    tensor of fa_block_mask_order_len(T) entries), for make_mask(tile_order=)."""
    import torch
    T = int(block_mask.shape[0])
    n = fa_block_mask_order_len(T)
    if n == 0 or block_mask.numel() != T * T:
        raise ValueError("expected a [T, T] block mask with 1 <= T <= 4096")
    out = torch.empty(n, dtype=torch.int32, device=block_mask.device)
    fa_block_mask_order(block_mask, T, causal, out, stream)
    return out


def fa_rope(q, k, q_out, k_out, B, Hq, Hk, N, d, rotary, layouts=None, stream=None):
    _check(lib.fa_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), B, Hq, Hk, N, d, rotary,
                       layouts, _stream(stream)), "fa_rope")


def fa_rope_bwd(dq_out, dk_out, dq, dk, B, Hq, Hk, N, d, rotary, layouts=None, stream=None):
    _check(lib.fa_rope_bwd(_ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), B, Hq, Hk, N, d,
                           rotary, layouts, _stream(stream)), "fa_rope_bwd")


def fa_rope_fp32(q, k, q_out, k_out, B, Hq, Hk, N, d, rotary, layouts=None, stream=None):
    _check(lib.fa_rope_fp32(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), B, Hq, Hk, N, d, rotary,
                            layouts, _stream(stream)), "fa_rope_fp32")


def fa_rope_bwd_fp32(dq_out, dk_out, dq, dk, B, Hq, Hk, N, d, rotary, layouts=None, stream=None):
    _check(lib.fa_rope_bwd_fp32(_ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), B, Hq, Hk, N, d,
                                rotary, layouts, _stream(stream)), "fa_rope_bwd_fp32")


def fa_cache_write(k, v, cache, start, q_len, B, T, rotary=None, layouts=None, stream=None):
    _check(lib.fa_cache_write(_ptr(k), _ptr(v), cache, _ptr(start), _ptr(q_len), B, T, rotary,
                              layouts, _stream(stream)), "fa_cache_write")


def fa_cache_read(cache, start, length, k, v, B, N, layouts=None, stream=None):
    _check(lib.fa_cache_read(cache, _ptr(start), _ptr(length), _ptr(k), _ptr(v), B, N, layouts,
                             _stream(stream)), "fa_cache_read")


def fa_cache_fwd_workspace_size(B, Hq, Hkv, T, d):
    return lib.fa_cache_fwd_workspace_size(B, Hq, Hkv, T, d)


def fa_cache_fwd(q, cache, start, q_len, tree_mask, o, lse, workspace, workspace_bytes, B, Hq, T,
                 scale, lq=None, lo=None, stream=None):
    _check(lib.fa_cache_fwd(_ptr(q), cache, _ptr(start), _ptr(q_len), _ptr(tree_mask), _ptr(o),
                            _ptr(lse), _ptr(workspace), workspace_bytes, B, Hq, T, scale, lq, lo,
                            _stream(stream)), "fa_cache_fwd")


def fa_status_string(code):
    return lib.fa_status_string(code).decode()


def fa_get_device_status(stream=None):
    """(status code, site) after synchronizing `stream`."""
    site = ctypes.c_int(0)
    code = lib.fa_get_device_status(_stream(stream), ctypes.byref(site))
    return code, site.value


def fa_debug_wait_timeout(limit_us, stream=None):
    _check(lib.fa_debug_wait_timeout(limit_us, _stream(stream)), "fa_debug_wait_timeout")


# ---------------------------------------------------------------------------
# conveniences: allocate outputs with torch, call the C functions
# ---------------------------------------------------------------------------

def _shape(q, *others):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d]")
    for t in others:
        if t.shape != q.shape or t.dtype != q.dtype or t.device != q.device:
            raise ValueError("every tensor must match q in shape, dtype and device")
    return tuple(int(x) for x in q.shape)


def forward(q, k, v, scale=None, causal=False, kv_len=None, block_mask=None, stream=None,
            dropout_p=0.0, seed=0, offset=0, bias=None, tile_order=None, rope=None,
            positions=None):
    """(O, lse) for CUDA tensors q, k, v [B,H,N,d] (bf16 or fp32) of any layout
    whose last dimension is contiguous; O takes q's layout where torch can
    keep it (torch.empty_like).  dropout_p > 0 drops attention probabilities
    (bf16 only); the backward needs the same dropout_p, seed and offset.
    bias: fp32 tensor broadcastable to [B, H, N, N] added to the scaled
    scores (bf16 only); the backward needs it too.  tile_order: the block
    mask's work order (block_mask_order), optional.  rope: q and k are rotated
    first (a Rope, at `positions`; without a stream the call then runs on torch's
    current stream); the backward takes the same, with the unrotated q and k."""
    import torch
    B, H, N, d = _shape(q, k, v)
    if rope is not None:
        with _on(stream, q.device):
            stream = torch.cuda.current_stream(q.device)
            q, k = _rope(lib.fa_rope, lib.fa_rope_fp32, q, k, rope, positions, None)
    scale = d ** -0.5 if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    mask = make_mask(kv_len, block_mask, tile_order=tile_order)
    opt = make_options(make_layouts(q=q, k=k, v=v, o=o), dropout_p, seed, offset,
                       None if bias is None else bias_of(bias))
    fn = fa_fwd_ex if q.dtype == torch.bfloat16 else fa_fwd_fp32_ex
    fn(q, k, v, o, lse, B, H, N, d, scale, causal, mask, opt, stream)
    return o, lse


def backward(q, k, v, o, do, lse, scale=None, causal=False, kv_len=None, block_mask=None,
             stream=None, workspace=None, dropout_p=0.0, seed=0, offset=0, bias=None,
             tile_order=None, rope=None, positions=None):
    """(dQ, dK, dV) for the forward above and output gradient do; each
    gradient takes the layout of its input where torch can keep it."""
    import torch
    B, H, N, d = _shape(q, k, v, o, do)
    if rope is not None:
        with _on(stream, q.device):
            stream = torch.cuda.current_stream(q.device)
            q, k = _rope(lib.fa_rope, lib.fa_rope_fp32, q, k, rope, positions, None)
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws_bytes = fa_bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    mask = make_mask(kv_len, block_mask, tile_order=tile_order)
    layouts = make_layouts(q=q, k=k, v=v, o=o, dO=do, dq=dq, dk=dk, dv=dv)
    opt = make_options(layouts, dropout_p, seed, offset, None if bias is None else bias_of(bias))
    fn = fa_bwd_ex if q.dtype == torch.bfloat16 else fa_bwd_fp32_ex
    fn(q, k, v, o, do, lse, dq, dk, dv, workspace, ws_bytes, B, H, N, d, scale, causal, mask,
       opt, stream)
    if rope is not None:
        with _on(stream, q.device):
            _rope(lib.fa_rope_bwd, lib.fa_rope_bwd_fp32, dq, dk, rope, positions, (dq, dk))
    return dq, dk, dv


# ---------------------------------------------------------------------------
# decoding: rotary positions, the key/value cache, attention over it.  Without
# a stream these run on torch's current stream of the tensors' device, with
# that device current for the call.
# ---------------------------------------------------------------------------

_NO_CONTEXT = contextlib.nullcontext()


def _on(stream, dev):
    """A context in which torch's current stream of `dev` is `stream` (a torch
    stream or a cudaStream_t as an int; None: as it is), so that what a call
    allocates belongs to the stream it runs on."""
    if stream is None:
        return _NO_CONTEXT
    import torch
    if not hasattr(stream, "cuda_stream"):
        stream = (torch.cuda.ExternalStream(int(stream), device=dev) if int(stream)
                  else torch.cuda.default_stream(dev))
    return torch.cuda.stream(stream)


_torch_c = None  # torch._C: imported by the first call (an import statement per call costs 0.3 us)


def _run(fn, dev, args, where):
    """fn(*args, stream) on torch's current stream of device index `dev`, with
    that device current."""
    global _torch_c
    if _torch_c is None:
        from torch import _C
        _torch_c = _C
    if _torch_c._cuda_getDevice() == dev:
        code = fn(*args, _torch_c._cuda_getCurrentRawStream(dev))
    else:
        import torch
        with torch.cuda.device(dev):
            code = fn(*args, _torch_c._cuda_getCurrentRawStream(dev))
    if code != 0:
        _check(code, where)


def _device(t, *others):
    """The CUDA device index that t and the others (None: skipped) are on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError("every tensor must be on cuda:%d" % dev)
    return dev


# What a call checks and works out from its tensors' shapes, strides and types alone,
# by these: a step of a decoding loop finds the step's before it.
_plans = {}


def _remember(key, plan):
    if len(_plans) >= 1024:
        _plans.clear()
    _plans[key] = plan
    return plan


def _layouts_of(kind, *tensors):
    """A `kind` (FaRopeLayouts, FaCacheLayouts, or FaLayout for one tensor) of the
    tensors' layouts."""
    ls = [FaLayout() if t is None else layout_of(t) for t in tensors]
    return ls[0] if kind is FaLayout else kind(*ls)


def _int32(name, t, *shape):
    import torch
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape %s" % (name, shape))


def rope_frequencies(dim, base=10000.0, scaling="none", factor=1.0, original=4096,
                     slow_turns=1.0, fast_turns=32.0, device="cuda"):
    """(frequencies, attention factor) of rotary positions over `dim` elements:
    f_p = base ** (-2 p / dim) radians per position, a float64 tensor of dim / 2
    (computed on the host), for Rope.  Scaling for contexts `factor` times
    longer than `original` positions:
      "none"    f_p
      "linear"  f_p / factor (positions interpolated)
      "base"    base times factor ** (dim / (dim - 2)): the fastest pair is
                kept, the slowest divided by factor
      "bands"   pairs with at least fast_turns turns over `original` positions
                keep f_p, those with at most slow_turns get f_p / factor, a
                linear ramp in the number of turns between; attention factor
                0.1 ln(factor) + 1
    """
    import math

    import torch
    if dim < 2 or dim % 2 or not factor > 0:
        raise ValueError("dim must be even and positive, factor positive")
    if scaling == "base":
        if dim < 4:
            raise ValueError('"base" scaling needs dim >= 4')
        base = base * factor ** (dim / (dim - 2.0))
    f = float(base) ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    attention = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        if not slow_turns < fast_turns:
            raise ValueError('"bands" scaling needs slow_turns < fast_turns')
        turns = original * f / (2.0 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        attention = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    elif scaling not in ("none", "base"):
        raise ValueError("unknown scaling %r" % (scaling,))
    return f.to(device), attention


class _Fixed:
    """Attributes are set once: the calls use pointers and sizes taken when the object is made."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError("a %s's %s is fixed: make another" % (type(self).__name__, name))
        self.__dict__[name] = value

    def __delattr__(self, name):
        raise AttributeError("a %s's %s is fixed" % (type(self).__name__, name))


class Rope(_Fixed):
    """Rotary positions: `freq`, a CUDA float64 tensor of dim / 2 radians per
    position (rope_frequencies), pairs (2p, 2p + 1) when interleaved, else
    (p, p + dim / 2), and a factor on the rotated elements."""

    def __init__(self, freq, interleaved=False, factor=1.0):
        import torch
        if freq.dim() != 1 or freq.dtype != torch.float64 or not freq.is_contiguous():
            raise ValueError("freq must be a contiguous 1-D float64 tensor")
        self.freq, self.dim, self._at = freq, 2 * freq.numel(), freq.data_ptr()
        self.interleaved, self.factor = bool(interleaved), float(factor)

    def struct(self, positions, B, N):
        """The FaRotary of a call over [B, N] tokens at `positions` (int32 [B, N]
        or [N], or None: the row index)."""
        return self._struct(positions, _position_stride(positions, B, N))

    def _struct(self, positions, stride):
        return FaRotary(self._at, None if positions is None else positions.data_ptr(), stride,
                        self.dim, self.interleaved, self.factor)


def _position_stride(positions, B, N):
    if positions is None:
        return 0
    import torch
    shape = positions.shape
    if (positions.dtype != torch.int32 or shape not in ((B, N), (N,))
            or (N > 1 and positions.stride(-1) != 1)):
        raise ValueError("positions must be int32 [B, N] or [N], contiguous along N")
    return positions.stride(0) if B > 1 and len(shape) == 2 else 0


def _rope_plan(q, k, qo, ko, positions):
    import torch
    B, Hq, N, d = q.shape if q.dim() == 4 else (0, 0, 0, 0)
    dt = q.dtype
    if not d or (dt is not torch.bfloat16 and dt is not torch.float32):
        raise ValueError("expected a bf16 or fp32 [B, H, N, d] tensor")
    Hk = 0
    if k is not None:
        Hk = k.shape[1] if k.dim() == 4 else 0
        if k.shape != (B, Hk, N, d) or k.dtype is not dt:
            raise ValueError("k must match q in dtype, batch, tokens and head dimension")
    if qo.shape != q.shape or qo.dtype is not dt or (k is None) != (ko is None) or (
            k is not None and (ko.shape != k.shape or ko.dtype is not dt)):
        raise ValueError("outputs must match their inputs in shape and dtype")
    return ((B, Hq, Hk, N, d), _layouts_of(FaRopeLayouts, q, k, qo, ko), dt is torch.bfloat16,
            _position_stride(positions, B, N))


def _rope(fn, fn32, q, k, rope, positions, out):
    if out is None:
        import torch
        out = torch.empty_like(q), None if k is None else torch.empty_like(k)
    qo, ko = out
    key = ("rope", q.shape, q.stride(), q.dtype, qo.shape, qo.stride(), qo.dtype,
           None if k is None else (k.shape, k.stride(), k.dtype),
           None if ko is None else (ko.shape, ko.stride(), ko.dtype),
           None if positions is None else (positions.shape, positions.stride(), positions.dtype))
    plan = _plans.get(key) or _remember(key, _rope_plan(q, k, qo, ko, positions))
    sizes, layouts, bf16, stride = plan
    dev = _device(q, k, qo, ko, rope.freq, positions)
    f = fn if bf16 else fn32
    _run(f, dev, (q.data_ptr(), None if k is None else k.data_ptr(), qo.data_ptr(),
                  None if ko is None else ko.data_ptr(), *sizes, rope._struct(positions, stride),
                  layouts), "fa_rope")
    return out


def rope(q, k, rope, positions=None, out=None, stream=None):
    """(q, k) [B, H, N, d] (bf16 or fp32, any layout with contiguous rows; k may
    be None and may have its own number of heads) rotated by their positions
    (int32 [B, N] or [N]; None: 0..N-1).  out: the tensors to write, which may be
    q and k themselves."""
    if stream is None:
        return _rope(lib.fa_rope, lib.fa_rope_fp32, q, k, rope, positions, out)
    with _on(stream, q.device):
        return _rope(lib.fa_rope, lib.fa_rope_fp32, q, k, rope, positions, out)


def rope_backward(dq, dk, rope, positions=None, out=None, stream=None):
    """The gradients of rope's inputs from those of its outputs."""
    if stream is None:
        return _rope(lib.fa_rope_bwd, lib.fa_rope_bwd_fp32, dq, dk, rope, positions, out)
    with _on(stream, dq.device):
        return _rope(lib.fa_rope_bwd, lib.fa_rope_bwd_fp32, dq, dk, rope, positions, out)


class KVCache(_Fixed):
    """A key/value cache (fa_cache) over the caller's CUDA tensors: k, v
    [pages, heads, page_size, d] (bf16, or float8_e4m3fn with fp32 scales
    [pages, heads, page_size]), and block_table, int32 [B, width] (None:
    sequence b owns page b).  The tensors are kept, and read and written where
    they are; their contents, the block table's too, may change between calls, the
    attributes may not."""

    def __init__(self, k, v, k_scale=None, v_scale=None, block_table=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise ValueError("k and v must match: [pages, heads, page_size, d]")
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("a cache is bf16 or float8_e4m3fn")
        e4m3 = k.dtype == torch.float8_e4m3fn
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("float8_e4m3fn caches, and only they, have k_scale and v_scale")
        for t in (v, k_scale, v_scale, block_table):
            if t is not None and t.device != k.device:
                raise ValueError("a cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.block_table = block_table
        pages, heads, page, d = k.shape
        scale_layout = None
        if e4m3:
            for s in (k_scale, v_scale):
                if (s.dtype != torch.float32 or s.shape != k.shape[:3]
                        or s.stride() != k_scale.stride() or (page > 1 and s.stride(2) != 1)):
                    raise ValueError("scales must be fp32 [pages, heads, page_size] with "
                                     "contiguous rows")
            scale_layout = FaLayout(k_scale.stride(0), k_scale.stride(1), 1)
        width, stride = 0, 0
        if block_table is not None:
            if (block_table.dim() != 2 or block_table.dtype != torch.int32
                    or (block_table.shape[1] > 1 and block_table.stride(1) != 1)):
                raise ValueError("block_table must be int32 [B, width] with contiguous rows")
            width = block_table.shape[1]
            stride = block_table.stride(0) if block_table.shape[0] > 1 else width
        self.format = FA_CACHE_E4M3 if e4m3 else FA_CACHE_BF16
        self.heads, self.d, self.device = heads, d, k.device
        self.sequences = pages if block_table is None else block_table.shape[0]
        self.capacity = page if block_table is None else width * page
        self._layout, self._scale_layout = layout_of(k), scale_layout
        self.struct = FaCache(
            self.format, pages, page, heads, d, k.data_ptr(), v.data_ptr(), _ptr(k_scale),
            _ptr(v_scale), ctypes.pointer(self._layout),
            ctypes.pointer(scale_layout) if e4m3 else None, _ptr(block_table), width, stride)

    @classmethod
    def empty(cls, pages, page_size, heads, d, dtype, block_table=None, device="cuda"):
        """A cache over newly allocated (uninitialised) tensors."""
        import torch
        k, v = (torch.empty(pages, heads, page_size, d, dtype=dtype, device=device)
                for _ in range(2))
        scales = (None, None)
        if dtype == torch.float8_e4m3fn:
            scales = tuple(torch.empty(pages, heads, page_size, dtype=torch.float32, device=device)
                           for _ in range(2))
        return cls(k, v, scales[0], scales[1], block_table)

    def _call(self, B, *tensors):
        """Checks a call over B sequences; its device index."""
        if B > self.sequences:
            raise ValueError("the cache has %d sequences, the call %d" % (self.sequences, B))
        return _device(self.k, *tensors)


def _dense_kv(cache, k, v, B, T):
    import torch
    shape = (B, cache.heads, T, cache.d)
    for t in (k, v):
        if t.dtype is not torch.bfloat16 or t.shape != shape:
            raise ValueError("k and v must be bf16 [B, heads, T, d]")
    return _layouts_of(FaCacheLayouts, k, v)


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _write_plan(cache, k, v, start, q_len, rope, positions):
    if k.dim() != 4:
        raise ValueError("k and v must be bf16 [B, heads, T, d]")
    B, _, T, _ = k.shape
    layouts = _dense_kv(cache, k, v, B, T)
    _int32("start", start, B)
    if q_len is not None:
        _int32("q_len", q_len, B)
    return B, T, layouts, 0 if rope is None else _position_stride(positions, B, T)


def cache_write(cache, k, v, start, q_len=None, rope=None, positions=None, stream=None):
    """Writes tokens t < q_len[b] of k, v (bf16 [B, heads, T, d]) to cache rows
    start[b] + t (start, q_len: int32 [B]).  rope: keys are rotated on the way, at
    `positions` (int32 [B, T] or [T]; None: the cache row)."""
    key = ("write", cache.heads, cache.d, k.shape, k.stride(), k.dtype, v.shape, v.stride(), v.dtype,
           start.shape, start.stride(), start.dtype, _meta(q_len), rope is None, _meta(positions))
    plan = _plans.get(key) or _remember(
        key, _write_plan(cache, k, v, start, q_len, rope, positions))
    B, T, layouts, stride = plan
    dev = cache._call(B, k, v, start, q_len, positions, None if rope is None else rope.freq)
    with _on(stream, cache.device):
        _run(lib.fa_cache_write, dev,
             (k.data_ptr(), v.data_ptr(), cache.struct, start.data_ptr(),
              None if q_len is None else q_len.data_ptr(), B, T,
              None if rope is None else rope._struct(positions, stride), layouts), "fa_cache_write")


def _read_plan(cache, n, start, length, k, v, B):
    for name, t in (("start", start), ("length", length)):
        if t is not None:
            _int32(name, t, B)
    return (_dense_kv(cache, k, v, B, n),)


def cache_read(cache, n, start=None, length=None, batch=None, out=None, stream=None):
    """(k, v) bf16 [B, heads, n, d]: rows start[b] .. start[b] + length[b] - 1 of
    every sequence (start None: 0, length None: n).  Rows from length[b] on are
    left as they were in `out`, and are zero without it."""
    B = next((int(t.shape[0]) for t in (start, length) if t is not None),
             batch if batch is not None else cache.sequences)
    with _on(stream, cache.device):
        if out is None:
            import torch
            out = tuple((torch.empty if length is None else torch.zeros)(
                (B, cache.heads, n, cache.d), dtype=torch.bfloat16, device=cache.device)
                for _ in range(2))
        k, v = out
        dev = cache._call(B, k, v, start, length)
        key = ("read", cache.heads, cache.d, n, B, k.shape, k.stride(), k.dtype, v.shape, v.stride(),
               v.dtype, _meta(start), _meta(length))
        plan = _plans.get(key) or _remember(key, _read_plan(cache, n, start, length, k, v, B))
        _run(lib.fa_cache_read, dev,
             (cache.struct, None if start is None else start.data_ptr(),
              None if length is None else length.data_ptr(), k.data_ptr(), v.data_ptr(), B, n,
              plan[0]), "fa_cache_read")
    return k, v


def tree_mask(parents, device="cuda"):
    """The int32 words [B, T, ceil(T/32)] of fa_cache_fwd's tree_mask from nested
    lists (or a CPU integer tensor) [B, T] of parents: token t descends from token
    parents[b][t] < t, or from the sequence itself where that is -1.  A token sees
    itself and its ancestors.  Built on the host."""
    import torch
    rows = [[int(p) for p in seq] for seq in parents]
    T = len(rows[0])
    words = torch.zeros(len(rows), T, (T + 31) // 32, dtype=torch.int64)
    for b, seq in enumerate(rows):
        if len(seq) != T:
            raise ValueError("every sequence needs T parents")
        seen = []
        for t, p in enumerate(seq):
            if not -1 <= p < t:
                raise ValueError("token %d has parent %d: expected -1 .. %d" % (t, p, t - 1))
            seen.append((seen[p] if p >= 0 else 0) | 1 << t)
            for w in range(words.shape[2]):
                words[b, t, w] = seen[t] >> 32 * w & 0xffffffff
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).to(device)


def _forward_plan(q, cache, start, q_len, tree_mask, o, lse):
    import torch
    B, Hq, T, d = q.shape
    if (o.shape != q.shape or o.dtype is not torch.bfloat16 or lse.dtype is not torch.float32
            or lse.shape != (B, Hq, T) or not lse.is_contiguous()):
        raise ValueError("o must match q, lse be contiguous fp32 [B, Hq, T]")
    _int32("start", start, B)
    if q_len is not None:
        _int32("q_len", q_len, B)
    if tree_mask is not None:
        _int32("tree_mask", tree_mask, B, T, (T + 31) // 32)
    return (B, Hq, T, lib.fa_cache_fwd_workspace_size(B, Hq, cache.heads, T, d),
            _layouts_of(FaLayout, q), _layouts_of(FaLayout, o))


def cache_forward(q, cache, start, q_len=None, tree_mask=None, scale=None, out=None,
                  workspace=None, stream=None):
    """(O, lse) of attention over the cache for new tokens q (bf16 [B, Hq, T, d],
    Hq a multiple of the cache's heads) whose own rows are cache rows start[b] + t
    (fa_cache_fwd).  tree_mask: int32 [B, T, ceil(T/32)] (None: each token sees the
    new tokens up to itself).  Rows t >= q_len[b] are left as they were in `out`,
    and are zero without it."""
    import torch
    if q.dim() != 4 or q.shape[3] != cache.d or q.dtype is not torch.bfloat16:
        raise ValueError("q must be bf16 [B, Hq, T, d] with the cache's d")
    with _on(stream, q.device):
        if out is None:
            new = torch.empty if q_len is None else torch.zeros
            out = ((torch.empty_like if q_len is None else torch.zeros_like)(q),
                   new(q.shape[:3], dtype=torch.float32, device=q.device))
        o, lse = out
        key = ("forward", cache.heads, q.shape, q.stride(), o.shape, o.stride(), o.dtype, lse.shape,
               lse.stride(), lse.dtype, start.shape, start.stride(), start.dtype, _meta(q_len),
               _meta(tree_mask))
        plan = _plans.get(key) or _remember(
            key, _forward_plan(q, cache, start, q_len, tree_mask, o, lse))
        B, Hq, T, bytes_, lq, lo = plan
        dev = cache._call(B, q, start, q_len, tree_mask, o, lse, workspace)
        if workspace is None:
            workspace = torch.empty(bytes_, dtype=torch.uint8, device=q.device)
        _run(lib.fa_cache_fwd, dev,
             (q.data_ptr(), cache.struct, start.data_ptr(),
              None if q_len is None else q_len.data_ptr(),
              None if tree_mask is None else tree_mask.data_ptr(), o.data_ptr(), lse.data_ptr(),
              workspace.data_ptr(), workspace.nbytes, B, Hq, T,
              cache.d ** -0.5 if scale is None else scale, lq, lo), "fa_cache_fwd")
    return o, lse


def decode_step(q, k, v, cache, start, q_len=None, tree_mask=None, rope=None, positions=None,
                scale=None, out=None, workspace=None, stream=None):
    """One decoding step: rotates q, writes the (rotated) k and v of the new
    tokens to cache rows start[b] + t, and attends over the cache; returns
    cache_forward's (O, lse).  With rope, positions are required (int32 [B, T] or
    [T]): a drafted token's position is its depth in the tree, not its row."""
    if rope is not None and positions is None:
        raise ValueError("rope needs the tokens' positions")
    with _on(stream, q.device):
        if rope is not None:
            q, _ = _rope(lib.fa_rope, lib.fa_rope_fp32, q, None, rope, positions, None)
        cache_write(cache, k, v, start, q_len, rope, positions)
        return cache_forward(q, cache, start, q_len, tree_mask, scale, out, workspace)
