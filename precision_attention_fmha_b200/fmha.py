"""ctypes binding of libfmha.so (include/fmha.h).

Argument marshalling only: every step of the computation runs in the CUDA
library. PyTorch supplies device memory (outputs are allocated with
``torch.empty``) and the current stream. If the library is missing the first
call raises -- there is no fallback implementation.

Tensors are token-major [B, S, H, D] with the last dim contiguous. 8-bit
operands are ``torch.int8`` (INT8) or ``torch.float8_e4m3fn`` (E4M3). A scale
factor is given as ``Scale(tensor, kind, rows_per_block)`` with ``kind`` one
of "per_tensor", "per_head", "per_token_block", "per_channel".
"""

import ctypes
import math
import os
import struct
from collections import namedtuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfmha.so")

BF16, FP16, FP32, E4M3, INT8 = 0, 1, 2, 3, 4
SF_KINDS = {None: 0, "none": 0, "per_tensor": 1, "per_head": 2, "per_token_block": 3, "per_channel": 4}
STATUS = {0: "FMHA_OK", 1: "FMHA_ERR_INVALID_ARG", 2: "FMHA_ERR_UNSUPPORTED", 3: "FMHA_ERR_CUDA",
          4: "FMHA_ERR_TIMEOUT", 5: "FMHA_ERR_DEVICE_INDEX"}
FMHA_OK, FMHA_ERR_INVALID_ARG, FMHA_ERR_UNSUPPORTED, FMHA_ERR_CUDA, FMHA_ERR_TIMEOUT, FMHA_ERR_DEVICE_INDEX = range(6)

Scale = namedtuple("Scale", ["tensor", "kind", "rows_per_block"], defaults=[0])


class FmhaError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class _Tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class _Sf(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("kind", ctypes.c_int32), ("rows_per_block", ctypes.c_int32)]


class _Args(ctypes.Structure):
    _fields_ = [("q", _Tensor), ("k", _Tensor), ("v", _Tensor), ("o", _Tensor),
                ("sf_q", _Sf), ("sf_k", _Sf), ("sf_v", _Sf), ("sf_p", _Sf),
                ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("Sq", ctypes.c_int32), ("Skv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("causal", ctypes.c_int32), ("lse", ctypes.c_void_p),
                ("p_terms", ctypes.c_int32), ("Dv", ctypes.c_int32), ("sf_o", _Sf)]


_lib = None


def load_library(path=None):
    """Loads libfmha.so once (raises if it is missing) and declares the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libfmha.so not built ({path}); run `python -m precision_attention_fmha_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.fmha_quantize_blockwise.argtypes = [ctypes.POINTER(_Tensor), ctypes.POINTER(_Tensor), ctypes.POINTER(_Sf),
                                            i32, i32, i32, i32, vp, sz, vp]
    lib.fmha_quantize_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.fmha_quantize_workspace_bytes.restype = sz
    lib.fmha_quantize_blockwise_shifted.argtypes = [ctypes.POINTER(_Tensor), vp, ctypes.POINTER(_Tensor),
                                                    ctypes.POINTER(_Sf), i32, i32, i32, i32, vp, sz, vp]
    lib.fmha_channel_mean.argtypes = [ctypes.POINTER(_Tensor), vp, i32, i32, i32, i32, vp, sz, vp]
    lib.fmha_channel_mean_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.fmha_channel_mean_workspace_bytes.restype = sz
    lib.fmha_fwd.argtypes = [ctypes.POINTER(_Args), vp]
    lib.fmha_fwd_block_sparse.argtypes = [ctypes.POINTER(_Args), vp, i64, i64, vp]
    lib.fmha_fwd_paged.argtypes = [ctypes.POINTER(_Args), vp, i32, i32, i32, vp, i64, i64, vp]
    lib.fmha_get_device_error.argtypes = [vp]
    lib.fmha_fwd_decode.argtypes = [ctypes.POINTER(_Args), vp, i32, i32, i32, vp, i64, i64, i32, vp, sz, vp]
    lib.fmha_quantize_nvfp4.argtypes = [vp, i64, i32, i32, vp, i64, vp, i64, vp, i32, vp]
    lib.fmha_decode_workspace_bytes.argtypes = [ctypes.POINTER(_Args), i32]
    lib.fmha_decode_workspace_bytes.restype = sz
    lib.fmha_decode_num_splits.argtypes = [ctypes.POINTER(_Args), i32]
    lib.fmha_decode_num_splits.restype = i32
    cache = vp  # packed fmha_cache_args (_CACHE_ARGS), or a pointer to a _CacheArgs
    lib.fmha_fwd_tree.argtypes = [cache, vp, i64, vp, sz, vp]
    lib.fmha_fwd_tree_workspace_bytes.argtypes = [cache]
    lib.fmha_fwd_selected.argtypes = [cache, vp, i32, i32, vp, sz, vp]
    lib.fmha_fwd_selected_workspace_bytes.argtypes = [cache, i32, i32]
    lib.fmha_key_bounds.argtypes = [cache, vp, i32, i32, vp, vp]
    lib.fmha_select_blocks.argtypes = [cache, vp, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.fmha_key_weights.argtypes = [cache, vp, i32, i32, i32, vp, sz, vp]
    lib.fmha_key_weights_workspace_bytes.argtypes = [cache, i32, i32]
    lib.fmha_evict_select.argtypes = [cache, vp, i32, i32, i32, i32, vp, vp, vp]
    lib.fmha_cache_compact.argtypes = [cache, cache, vp, i64, i64, i32, vp, vp, vp, i32, vp, i32, vp]
    for f in ("fmha_fwd_tree_workspace_bytes", "fmha_fwd_selected_workspace_bytes", "fmha_key_weights_workspace_bytes"):
        getattr(lib, f).restype = sz
    lib.fmha_status_string.argtypes = [ctypes.c_int]
    lib.fmha_status_string.restype = ctypes.c_char_p
    lib.fmha_last_error_message.restype = ctypes.c_char_p
    lib.fmha_set_wait_timeout_cycles.argtypes = [ctypes.c_uint64]
    for f in ("fmha_quantize_blockwise", "fmha_fwd", "fmha_fwd_block_sparse", "fmha_fwd_paged",
              "fmha_get_device_error", "fmha_quantize_blockwise_shifted", "fmha_channel_mean"):
        getattr(lib, f).restype = ctypes.c_int
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(status):
    if status != 0:
        msg = load_library().fmha_last_error_message().decode()
        raise FmhaError(status, msg)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return FP16
    if t.dtype == torch.float8_e4m3fn:
        return E4M3
    if t.dtype == torch.int8:
        return INT8
    raise TypeError(f"unsupported dtype {t.dtype}")


def _tensor(t):
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError("expected a [B, S, H, D] tensor with a contiguous last dim")
    return _Tensor(t.data_ptr(), _dtype_code(t), 0, t.stride(0), t.stride(1), t.stride(2))


def _sf(s):
    if s is None:
        return _Sf(None, 0, 0)
    if not isinstance(s, Scale):
        raise TypeError("scale factors are Scale(tensor, kind, rows_per_block)")
    if s.tensor.dtype != torch.float32 or not s.tensor.is_contiguous():
        raise ValueError("scale tensors must be contiguous float32")
    return _Sf(s.tensor.data_ptr(), SF_KINDS[s.kind], int(s.rows_per_block or 0))


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def quantize_workspace_bytes(kind, B, S, H, D):
    return load_library().fmha_quantize_workspace_bytes(SF_KINDS[kind], B, S, H, D)


def scale_shape(kind, B, S, H, D, rows_per_block=None):
    if kind == "per_tensor":
        return (1,)
    if kind == "per_head":
        return (B, H)
    if kind == "per_token_block":
        return (B, H, math.ceil(S / rows_per_block))
    if kind == "per_channel":
        return (B, H, D)
    raise ValueError(kind)


def fmha_quantize_blockwise(x, out_dtype, kind, rows_per_block=None, out=None, scales=None, workspace=None,
                            stream=None, shift=None):
    """BF16 x [B,S,H,D] -> (codes, fp32 scales). out_dtype: torch.int8 or torch.float8_e4m3fn.

    shift (optional, contiguous fp32 [B, H, D] on the device): quantize
    x - shift instead of x (K smoothing; see ``channel_mean``).
    """
    lib = load_library()
    if shift is not None and (shift.dtype != torch.float32 or not shift.is_contiguous()
                              or tuple(shift.shape) != (x.shape[0], x.shape[2], x.shape[3])):
        raise ValueError("shift must be a contiguous float32 [B, H, D] tensor")
    B, S, H, D = x.shape
    if out is None:
        out = torch.empty((B, S, H, D), dtype=out_dtype, device=x.device)
    if scales is None:
        scales = torch.empty(scale_shape(kind, B, S, H, D, rows_per_block), dtype=torch.float32, device=x.device)
    need = lib.fmha_quantize_workspace_bytes(SF_KINDS[kind], B, S, H, D)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    src, dst = _tensor(x), _tensor(out)
    sf = _Sf(scales.data_ptr(), SF_KINDS[kind], int(rows_per_block or 0))
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if shift is None:
        _check(lib.fmha_quantize_blockwise(ctypes.byref(src), ctypes.byref(dst), ctypes.byref(sf), B, S, H, D,
                                           ws_ptr, ws_bytes, _stream(stream)))
    else:
        _check(lib.fmha_quantize_blockwise_shifted(ctypes.byref(src), shift.data_ptr(), ctypes.byref(dst),
                                                   ctypes.byref(sf), B, S, H, D, ws_ptr, ws_bytes, _stream(stream)))
    return out, scales


def channel_mean_workspace_bytes(B, S, H, D):
    return load_library().fmha_channel_mean_workspace_bytes(B, S, H, D)


def channel_mean(x, out=None, workspace=None, stream=None):
    """Token mean per (b, h, d) of BF16 x [B, S, H, D] -> fp32 [B, H, D] (fp64 sums)."""
    lib = load_library()
    B, S, H, D = x.shape
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.float32, device=x.device)
    need = lib.fmha_channel_mean_workspace_bytes(B, S, H, D)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    src = _tensor(x)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.fmha_channel_mean(ctypes.byref(src), out.data_ptr(), B, S, H, D, ws_ptr, ws_bytes,
                                 _stream(stream)))
    return out


def quantize_smoothed(x, out_dtype, kind, rows_per_block=None, stream=None):
    """SageAttention K smoothing: (codes, scales, mean) with codes * scales ~= x - mean."""
    mean = channel_mean(x, stream=stream)
    codes, scales = fmha_quantize_blockwise(x, out_dtype, kind, rows_per_block, stream=stream, shift=mean)
    return codes, scales, mean


def _args(q, k, v, out, sf_q, sf_k, sf_v, sf_p, softmax_scale, causal, lse, Skv=None, p_terms=1, sf_o=None):
    B, Sq, Hq, D = q.shape
    Hkv = k.shape[2]
    a = _Args()
    a.q, a.k, a.v, a.o = _tensor(q), _tensor(k), _tensor(v), _tensor(out)
    a.sf_q, a.sf_k, a.sf_v, a.sf_p = _sf(sf_q), _sf(sf_k), _sf(sf_v), _sf(sf_p)
    a.B, a.Hq, a.Hkv, a.Sq, a.Skv, a.D = B, Hq, Hkv, Sq, k.shape[1] if Skv is None else Skv, D
    a.softmax_scale = float(softmax_scale) if softmax_scale else 0.0
    a.causal = 1 if causal else 0
    a.lse = lse.data_ptr() if lse is not None else None
    a.p_terms = int(p_terms)
    a.Dv = v.shape[3]
    a.sf_o = _sf(sf_o)
    return a


def _out_like(q, v, out):
    """O is [B, Sq, Hq, Dv]: Dv, the head dim of V, differs from q's for D = 192 / 128."""
    if out is None:
        out = torch.empty(q.shape[:3] + v.shape[3:], dtype=torch.bfloat16, device=q.device)
    return out


def fmha_fwd(q, k, v, out=None, sf_q=None, sf_k=None, sf_v=None, sf_p=None, softmax_scale=None, causal=False,
             lse=None, stream=None, p_terms=1, sf_o=None):
    """Dense attention. Returns O (BF16 [B, Sq, Hq, Dv]). p_terms=2 splits an E4M3 P into two terms.

    Head dims: q / k D and v / out Dv, equal (64 or 128), or D = 192 with Dv = 128.

    An E4M3 ``out`` (torch.float8_e4m3fn, D = 128) receives E4M3(O / sf_o),
    with sf_o an optional per-tensor Scale (1.0 when None)."""
    lib = load_library()
    out = _out_like(q, v, out)
    a = _args(q, k, v, out, sf_q, sf_k, sf_v, sf_p, softmax_scale, causal, lse, p_terms=p_terms, sf_o=sf_o)
    _check(lib.fmha_fwd(ctypes.byref(a), _stream(stream)))
    return out


def fmha_fwd_block_sparse(q, k, v, mask, out=None, sf_q=None, sf_k=None, sf_v=None, sf_p=None,
                          softmax_scale=None, causal=False, lse=None, stream=None, p_terms=1, sf_o=None):
    """Attention restricted by a uint8 128x128 block mask [B or 1, Hkv or 1, ceil(Sq/128), ceil(Skv/128)]."""
    lib = load_library()
    out = _out_like(q, v, out)
    a = _args(q, k, v, out, sf_q, sf_k, sf_v, sf_p, softmax_scale, causal, lse, p_terms=p_terms, sf_o=sf_o)
    msb, msh = _mask_strides(mask, q.shape[1], k.shape[1])
    _check(lib.fmha_fwd_block_sparse(ctypes.byref(a), mask.data_ptr(), msb, msh, _stream(stream)))
    return out


def _mask_strides(mask, Sq, Skv):
    if mask.dtype != torch.uint8 or mask.dim() != 4:
        raise ValueError("mask must be uint8 [B, Hkv, ceil(Sq/128), ceil(Skv/128)]")
    nq, nk = math.ceil(Sq / 128), math.ceil(Skv / 128)
    if mask.shape[2] != nq or mask.shape[3] != nk or mask.stride(3) != 1 or mask.stride(2) != nk:
        raise ValueError(f"mask inner dims must be contiguous [{nq}, {nk}]")
    return (mask.stride(0) if mask.shape[0] > 1 else 0), (mask.stride(1) if mask.shape[1] > 1 else 0)


def fmha_fwd_paged(q, k_pool, v_pool, page_table, Skv, mask=None, out=None, sf_q=None, sf_k=None, sf_v=None,
                   sf_p=None, softmax_scale=None, causal=False, lse=None, stream=None, p_terms=1, sf_o=None):
    """Attention over a paged K/V pool [num_pages, page_size, Hkv, D] through page_table int32 [B, max_pages]."""
    lib = load_library()
    out = _out_like(q, v_pool, out)
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
        raise ValueError("page_table must be contiguous int32 [B, max_pages_per_seq]")
    a = _args(q, k_pool, v_pool, out, sf_q, sf_k, sf_v, sf_p, softmax_scale, causal, lse, Skv=Skv, p_terms=p_terms,
              sf_o=sf_o)
    mptr, msb, msh = None, 0, 0
    if mask is not None:
        msb, msh = _mask_strides(mask, q.shape[1], Skv)
        mptr = mask.data_ptr()
    _check(lib.fmha_fwd_paged(ctypes.byref(a), page_table.data_ptr(), k_pool.shape[0], k_pool.shape[1],
                              page_table.shape[1], mptr, msb, msh, _stream(stream)))
    return out


def fmha_fwd_decode(q, k, v, page_table=None, Skv=None, mask=None, num_splits=0, workspace=None, out=None,
                    sf_q=None, sf_k=None, sf_v=None, sf_p=None, softmax_scale=None, causal=False, lse=None,
                    stream=None):
    """Decode-shaped attention (few query tokens, GQA-packed tiles, split-KV).

    k / v: contiguous [B, Skv, Hkv, D], or page pools [num_pages, page_size, Hkv, D]
    with page_table int32 [B, max_pages] and Skv. The workspace (uint8 CUDA tensor)
    is allocated here when not given. Returns O (BF16 [B, Sq, Hq, D])."""
    lib = load_library()
    out = _out_like(q, v, out)
    if page_table is not None:
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
            raise ValueError("page_table must be contiguous int32 [B, max_pages_per_seq]")
        if Skv is None:
            raise ValueError("Skv is required with a page table")
    a = _args(q, k, v, out, sf_q, sf_k, sf_v, sf_p, softmax_scale, causal, lse, Skv=Skv)
    mptr, msb, msh = None, 0, 0
    if mask is not None:
        msb, msh = _mask_strides(mask, q.shape[1], a.Skv)
        mptr = mask.data_ptr()
    need = lib.fmha_decode_workspace_bytes(ctypes.byref(a), int(num_splits))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wptr, wbytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None \
        else (None, 0)
    if page_table is not None:
        pt, npages, psize, maxp = page_table.data_ptr(), k.shape[0], k.shape[1], page_table.shape[1]
    else:
        pt, npages, psize, maxp = None, 0, 0, 0
    _check(lib.fmha_fwd_decode(ctypes.byref(a), pt, npages, psize, maxp, mptr, msb, msh, int(num_splits), wptr,
                               wbytes, _stream(stream)))
    return out


def decode_num_splits(q, k, Skv=None, num_splits=0):
    """KV splits fmha_fwd_decode uses for these shapes (host only)."""
    B, Sq, Hq, D = q.shape
    a = _Args()
    a.B, a.Hq, a.Hkv, a.Sq, a.Skv, a.D = B, Hq, k.shape[2], Sq, k.shape[1] if Skv is None else Skv, D
    return load_library().fmha_decode_num_splits(ctypes.byref(a), int(num_splits))


def quantize_nvfp4(x, fast_math=False, codes=None, block_scales=None, token_scales=None, stream=None):
    """Per-token NVFP4 of a BF16 CUDA matrix [rows, K] (row stride x.stride(0)).

    Returns (codes uint8 [rows, K/2], block_scales float8_e4m3fn [rows, K/16],
    token_scales float32 [rows])."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a BF16 [rows, K] matrix with unit column stride")
    rows, K = x.shape
    dev = x.device
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev) if codes is None else codes
    block_scales = torch.empty((rows, K // 16), dtype=torch.uint8, device=dev) if block_scales is None \
        else block_scales.view(torch.uint8)
    token_scales = torch.empty((rows,), dtype=torch.float32, device=dev) if token_scales is None else token_scales
    _check(load_library().fmha_quantize_nvfp4(x.data_ptr(), x.stride(0), rows, K, codes.data_ptr(), codes.stride(0),
                                              block_scales.data_ptr(), block_scales.stride(0),
                                              token_scales.data_ptr(), 1 if fast_math else 0, _stream(stream)))
    return codes, block_scales.view(torch.float8_e4m3fn), token_scales


def decode_workspace_bytes(q, k, Skv=None, num_splits=0):
    """Workspace bytes fmha_fwd_decode needs for these shapes (host only)."""
    B, Sq, Hq, D = q.shape
    a = _Args()
    a.B, a.Hq, a.Hkv, a.Sq, a.Skv, a.D = B, Hq, k.shape[2], Sq, k.shape[1] if Skv is None else Skv, D
    return load_library().fmha_decode_workspace_bytes(ctypes.byref(a), int(num_splits))


def decode_num_parts(q, k, Skv=None, num_splits=0):
    """Partial outputs fmha_fwd_decode merges (1: no merge launch)."""
    need = decode_workspace_bytes(q, k, Skv, num_splits)
    if need == 0:
        return 1
    B, Sq, Hq, D = q.shape
    return (need - 16) // (B * Sq * Hq * (D + 1) * 4)


def get_device_error(stream=None):
    """Synchronises the stream and raises FmhaError if a kernel recorded a device-side error."""
    _check(load_library().fmha_get_device_error(_stream(stream)))


def set_wait_timeout_cycles(cycles):
    load_library().fmha_set_wait_timeout_cycles(int(cycles))


# ------------------------------------------------- operators over a ragged cache
class _CacheArgs(ctypes.Structure):
    _fields_ = [("q", _Tensor), ("k", _Tensor), ("v", _Tensor), ("o", _Tensor), ("sf_k", _Sf), ("sf_v", _Sf),
                ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("lens", ctypes.c_void_p), ("q_lens", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("lse", ctypes.c_void_p)]


# The same layout as packed values: one call fills the 45 members, where setting them one by one in the structure
# took 16 us of a decoding step's host time (packed: 5 us).
_NO_TABLE = (0, 0, 0, 0)
_CACHE_ARGS = struct.Struct("@" + 4 * "Pii3q" + 2 * "Pii" + "6i3P3ifP")


def _pack(*fields):
    try:
        return _CACHE_ARGS.pack(*fields)
    except struct.error as e:
        raise ValueError(f"a size of the cache or the queries is out of range: {e}") from None


def _int32s(what, *values):
    """Checks that 32-bit arguments hold the values (ctypes would drop their higher bits)."""
    for x in values:
        if not -0x80000000 <= x < 0x80000000:
            raise ValueError(f"{what} {values}: a number is out of range")


_NO_TENSOR, _NO_SF = (0, 0, 0, 0, 0, 0), (0, 0, 0)
_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float8_e4m3fn: E4M3, torch.int8: INT8}


class _launch:
    """Makes the tensors' device current, and `stream` (None: that device's current stream) the stream that
    outputs and workspaces allocated inside belong to. Entering gives the stream handle."""

    __slots__ = ("contexts", "stream", "device")

    def __init__(self, stream, first, *tensors):
        device = first.get_device()
        for t in tensors:
            if t is not None and t.get_device() != device:
                device = -1
        if device < 0:
            raise ValueError("all tensors must be on one CUDA device, got "
                             f"{sorted({str(t.device) for t in (first, *tensors) if t is not None})}")
        if stream is not None and stream.device.index != device:
            raise ValueError(f"stream of {stream.device} for tensors of cuda:{device}")
        self.stream, self.device, self.contexts = stream, device, ()

    def __enter__(self):
        if self.device != torch.cuda.current_device():
            self.contexts += (torch.cuda.device(self.device),)
        if self.stream is None:
            if not self.contexts:
                return _raw_stream(self.device)
        else:
            self.contexts += (torch.cuda.stream(self.stream),)
        for c in self.contexts:
            c.__enter__()
        return _raw_stream(self.device)

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _raw_stream(device):
    """Handle of the device's current stream (a tenth of the time that making a torch Stream takes)."""
    return torch._C._cuda_getCurrentRawStream(device)


def _array(t, dtype, shape, what):
    """Checks a tensor's type, shape and contiguity; returns its address (0 for None)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {list(shape)}")
    return t.data_ptr()


def _ints(t, shape, what):
    return _array(t, torch.int32, shape, what)


def _floats(t, shape, what):
    return _array(t, torch.float32, shape, what)


def _packed(t):
    stride = t.stride()
    if len(stride) != 4 or stride[3] != 1:
        raise ValueError("expected a [B, S, H, D] tensor with a contiguous last dim")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return (t.data_ptr(), code, 0, stride[0], stride[1], stride[2])


def _cache_sf(s, B, Hkv, what):
    if s is None:
        return _NO_SF
    sf = _sf(s)
    if s.kind == "per_head" and tuple(s.tensor.shape) != (B, Hkv):
        raise ValueError(f"{what}: per-head scales must have shape [{B}, {Hkv}]")
    if s.kind not in (None, "none") and s.tensor.numel() == 0:
        raise ValueError(f"{what}: empty scale tensor")
    return (sf.ptr or 0, sf.kind, sf.rows_per_block)


def _cache_view(k, v, page_table):
    """The tensor fields of k and v, and B, Hkv, D, capacity and the page table's fields."""
    tk = _packed(k)
    shape = k.shape
    n, rows, Hkv, D = shape
    tv = _NO_TENSOR
    if v is not None:
        if v.shape != shape:
            raise ValueError(f"k {list(shape)} and v {list(v.shape)} differ in shape")
        tv = _packed(v)
    if page_table is None:
        return tk, tv, n, Hkv, D, rows, _NO_TABLE
    pages = page_table.shape
    if len(pages) != 2:
        raise ValueError("page_table must be contiguous int32 [B, max_pages_per_seq]")
    B, per = pages
    return tk, tv, B, Hkv, D, per * rows, (_array(page_table, torch.int32, pages, "page_table"), n, rows, per)


def _cache_args(k, lens, page_table, q=None, v=None, out=None, q_lens=None, sf_k=None, sf_v=None,
                softmax_scale=None, lse=None):
    """fmha_cache_args of k (and v) [B, S, Hkv, D], or pools [pages, page_size, Hkv, D] with a page table
    [B, max_pages]; and (B, Hkv, D, capacity)."""
    tk, tv, B, Hkv, D, capacity, table = _cache_view(k, v, page_table)
    tq = to = _NO_TENSOR
    T = Hq = lse_ptr = 0
    if q is not None:
        tq = _packed(q)
        q_shape = q.shape
        q_B, T, Hq, q_D = q_shape
        if q_B != B or q_D != D:
            raise ValueError(f"q {list(q_shape)} does not fit a cache of {B} sequences with head dim {D}")
        if lse is not None:
            lse_ptr = _array(lse, torch.float32, (B, Hq, T), "lse")
        if out is not None:
            if out.shape != q_shape:
                raise ValueError(f"out {list(out.shape)} differs from q {list(q_shape)} in shape")
            to = _packed(out)
    args = _pack(*tq, *tk, *tv, *to, *_cache_sf(sf_k, B, Hkv, "sf_k"), *_cache_sf(sf_v, B, Hkv, "sf_v"),
                 B, T, Hq, Hkv, D, capacity, _array(lens, torch.int32, (B,), "lens"),
                 _array(q_lens, torch.int32, (B,), "q_lens"), *table,
                 float(softmax_scale) if softmax_scale else 0.0, lse_ptr)
    return args, (B, Hkv, D, capacity)


def _scratch(workspace, need, q):
    """The caller's workspace, or one allocated here; its address and size."""
    if workspace is None:
        if need == 0:
            return None, 0, 0
        workspace = q.new_empty(need, dtype=torch.uint8)
    elif workspace.get_device() != q.get_device():
        raise ValueError(f"workspace on {workspace.device}, tensors on {q.device}")
    elif not workspace.is_contiguous():  # an expanded one claims more bytes than it has
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _sf_tensors(*scales):
    return [s.tensor for s in scales if s is not None]


def fmha_fwd_tree(q, k, v, ctx_lens, tree_mask=None, tree_lens=None, page_table=None, workspace=None, out=None,
                  sf_k=None, sf_v=None, softmax_scale=None, lse=None, stream=None):
    """Attention of a tree of drafted tokens over a ragged cache. Returns O (BF16 [B, T, Hq, D]).

    q: BF16 [B, T, Hq, D], the drafted nodes. k / v: [B, S, Hkv, D], or page pools
    [num_pages, page_size, Hkv, D] with page_table int32 [B, max_pages]; BF16 or E4M3 (with sf_k / sf_v).
    ctx_lens: int32 [B], tokens before the tree; node j of sequence b stands at position ctx_lens[b] + j.
    tree_lens: int32 [B], nodes in use (None: T). tree_mask: uint8 [B or 1, T, T], nonzero where node i (row)
    sees node j; None: a chain (node i sees nodes 0..i), so T = 1 is an ordinary decoding step of a ragged batch.
    lse (optional): contiguous fp32 [B, Hq, T]. Rows that see no key give O = 0, lse = -inf."""
    T = q.shape[1] if q.dim() == 4 else 0
    mask, mask_sb = 0, 0
    if tree_mask is not None:
        st = tree_mask.stride()
        if (tree_mask.dtype != torch.uint8 or len(st) != 3 or tree_mask.shape[0] not in (1, q.shape[0])
                or tree_mask.shape[1:] != (T, T) or (T > 1 and st[1:] != (T, 1))):
            raise ValueError(f"tree_mask must be uint8 [{q.shape[0]} or 1, {T}, {T}] with contiguous rows")
        mask, mask_sb = tree_mask.data_ptr(), st[0] if tree_mask.shape[0] > 1 else 0
    lib = load_library()
    with _launch(stream, q, k, v, ctx_lens, tree_mask, tree_lens, page_table, out, lse, *_sf_tensors(sf_k, sf_v)) as s:
        out = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else out
        a, _ = _cache_args(k, ctx_lens, page_table, q=q, v=v, out=out, q_lens=tree_lens, sf_k=sf_k, sf_v=sf_v,
                           softmax_scale=softmax_scale, lse=lse)
        workspace, ptr, size = _scratch(workspace, lib.fmha_fwd_tree_workspace_bytes(a), q)
        _check(lib.fmha_fwd_tree(a, mask, mask_sb, ptr, size, s))
    return out


def tree_workspace_bytes(q, k, page_table=None):
    """Workspace bytes fmha_fwd_tree needs for these shapes (host only)."""
    lens = torch.empty(q.shape[0], dtype=torch.int32)
    return load_library().fmha_fwd_tree_workspace_bytes(_cache_args(k, lens, page_table, q=q)[0])


def fmha_fwd_selected(q, k, v, blocks, lens, block, q_lens=None, page_table=None, workspace=None, out=None,
                      sf_k=None, sf_v=None, softmax_scale=None, lse=None, stream=None):
    """Attention over the key blocks picked for each query token. Returns O (BF16 [B, T, Hq, D]).

    blocks: contiguous int32 [B, T, Hkv, top], ids of the `block`-key blocks (16, 32, 64 or 128) that query token
    t reads in KV head h; negative: none (``select_blocks`` makes them). lens: int32 [B], tokens in the cache;
    the q_lens[b] (None: T) query tokens are its last ones, and each sees keys up to its own position."""
    if blocks.dim() != 4:
        raise ValueError("blocks must be a contiguous int32 [B, T, Hkv, top] tensor")
    top, block = blocks.shape[3], int(block)
    _int32s("top, block", top, block)
    ids = _ints(blocks, (q.shape[0], q.shape[1], k.shape[2], top), "blocks")
    lib = load_library()
    with _launch(stream, q, k, v, blocks, lens, q_lens, page_table, out, lse, *_sf_tensors(sf_k, sf_v)) as s:
        out = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else out
        a, _ = _cache_args(k, lens, page_table, q=q, v=v, out=out, q_lens=q_lens, sf_k=sf_k, sf_v=sf_v,
                           softmax_scale=softmax_scale, lse=lse)
        workspace, ptr, size = _scratch(workspace, lib.fmha_fwd_selected_workspace_bytes(a, top, block), q)
        _check(lib.fmha_fwd_selected(a, ids, top, block, ptr, size, s))
    return out


def key_bounds(k, lens, block, page_table=None, bounds=None, start=None, stream=None):
    """Smallest and largest key of each `block`-key block (16, 32, 64 or 128) and channel.

    k: [B, S, Hkv, D], or a page pool with page_table; lens: int32 [B], tokens in the cache. Returns bounds BF16
    [B, Hkv, n_blocks, 2, D] (minima, maxima); blocks past a sequence's end are left as they were (zeros when
    allocated here). start: int32 [B]: blocks that end at or before it are left, so that a step refreshes the
    newest block only."""
    block = int(block)
    a, (B, Hkv, D, capacity) = _cache_args(k, lens, page_table)
    if bounds is None:
        shape = (B, Hkv, -(-capacity // block) if block > 0 else 0, 2, D)
    else:
        shape = tuple(bounds.shape)
        if (bounds.dtype != torch.bfloat16 or len(shape) != 5 or shape[:2] != (B, Hkv) or shape[3:] != (2, D)
                or not bounds.is_contiguous()):
            raise ValueError(f"bounds must be contiguous BF16 [{B}, {Hkv}, n_blocks, 2, {D}]")
    start_ptr = _ints(start, (B,), "start")
    _int32s("n_blocks, block", shape[2], block)
    lib = load_library()
    with _launch(stream, k, lens, page_table, bounds, start) as s:
        if bounds is None:
            bounds = torch.zeros(shape, dtype=torch.bfloat16, device=k.device)
        _check(lib.fmha_key_bounds(a, bounds.data_ptr(), shape[2], block, start_ptr, s))
    return bounds


def select_blocks(q, bounds, lens, block, top, sink_blocks=0, recent_blocks=1, q_lens=None, q_tile=1, out=None,
                  stream=None):
    """Picks the blocks of keys that each query attends to, by the score sum_h sum_d max(q_hd min_jd, q_hd max_jd).

    q: BF16 [B, T, Hq, D], the last q_lens[b] (None: T) of the lens[b] tokens; bounds as from ``key_bounds``. The
    first sink_blocks and the last recent_blocks in sight are picked first, then the best scores, up to `top`.
    q_tile 1: int32 [B, T, Hkv, top], ascending ids then -1, for ``fmha_fwd_selected``. q_tile 128 (block 128):
    the uint8 mask [B, Hkv, ceil(T/128), n_blocks] of ``fmha_fwd_block_sparse`` / ``fmha_fwd_paged``, picked by
    tiles of 128 query tokens."""
    shape, q_shape = bounds.shape, q.shape
    if (bounds.dtype != torch.bfloat16 or len(shape) != 5 or shape[3] != 2 or not bounds.is_contiguous()
            or len(q_shape) != 4 or shape[0] != q_shape[0] or shape[4] != q_shape[3]):
        raise ValueError("bounds must be contiguous BF16 [B, Hkv, n_blocks, 2, D] for q [B, T, Hq, D]")
    B, T, Hq, D = q_shape
    Hkv, n_blocks = shape[1], shape[2]
    block, top, q_tile, sink_blocks, recent_blocks = int(block), int(top), int(q_tile), int(sink_blocks), int(recent_blocks)
    _int32s("n_blocks, block, top, q_tile, sink_blocks, recent_blocks", n_blocks, block, top, q_tile, sink_blocks, recent_blocks)
    a = _pack(*_packed(q), *_NO_TENSOR, *_NO_TENSOR, *_NO_TENSOR, *_NO_SF, *_NO_SF, B, T, Hq, Hkv, D, 0,
              _ints(lens, (B,), "lens"), _ints(q_lens, (B,), "q_lens"), *_NO_TABLE, 0.0, 0)
    shape, dtype = ((B, T, Hkv, top), torch.int32) if q_tile == 1 else ((B, Hkv, -(-T // 128), n_blocks), torch.uint8)
    _array(out, dtype, shape, "out")
    lib = load_library()
    with _launch(stream, q, bounds, lens, q_lens, out) as s:
        if out is None:
            out = q.new_empty(shape if top >= 0 else 0, dtype=dtype)
        _check(lib.fmha_select_blocks(a, bounds.data_ptr(), n_blocks, block, top, sink_blocks,
                                      recent_blocks, q_tile, out.data_ptr(), s))
    return out


def key_weights(q, k, lse, weights, lens, q_lens=None, page_table=None, causal=True, accumulate=True,
                sf_k=None, softmax_scale=None, workspace=None, stream=None):
    """Adds (accumulate=False: writes) to weights fp32 [B, Hkv, n] the attention weight each key gathers over q.

    weights[b, h, s] (+)= sum_t sum_g exp(scale * q_tg . k_s - lse[b, g, t]), over the query heads g of KV head h
    and the tokens t that see key s. lse: contiguous fp32 [B, Hq, T] of the attention call on the same q and keys.
    q holds the last q_lens[b] (None: T) of the lens[b] tokens. Entries past lens[b] are left as they were."""
    a, (B, Hkv, _, _) = _cache_args(k, lens, page_table, q=q, q_lens=q_lens, sf_k=sf_k, softmax_scale=softmax_scale, lse=lse)
    if weights.dim() != 3:
        raise ValueError("weights must be a contiguous float32 [B, Hkv, n] tensor")
    w = _floats(weights, (B, Hkv, weights.shape[2]), "weights")
    _int32s("n", weights.shape[2])
    lib = load_library()
    with _launch(stream, q, k, lse, weights, lens, q_lens, page_table, *_sf_tensors(sf_k)) as s:
        n, causal = weights.shape[2], 1 if causal else 0
        workspace, ptr, size = _scratch(workspace, lib.fmha_key_weights_workspace_bytes(a, n, causal), q)
        _check(lib.fmha_key_weights(a, w, n, causal, 1 if accumulate else 0, ptr, size, s))
    return weights


def evict_select(weights, lens, budget, sinks=0, recent=0, keep=None, counts=None, stream=None):
    """The positions that stay in the cache of each (sequence, KV head) under `budget` keys.

    weights: contiguous fp32 [B, Hkv, n]; lens: int32 [B]. Returns (keep int32 [B, Hkv, budget]: ascending positions,
    then -1; counts int32 [B]: min(lens, budget)). The first `sinks` and last `recent` positions always stay, then
    the largest weights, ties to the lowest position."""
    if weights.dim() != 3:
        raise ValueError("weights must be a contiguous float32 [B, Hkv, n] tensor")
    B, Hkv, n = weights.shape
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    _int32s("n, budget, sinks, recent", n, budget, sinks, recent)
    a = _pack(*_NO_TENSOR, *_NO_TENSOR, *_NO_TENSOR, *_NO_TENSOR, *_NO_SF, *_NO_SF, B, 0, 0, Hkv, 0, 0,
              _ints(lens, (B,), "lens"), 0, *_NO_TABLE, 0.0, 0)
    w = _floats(weights, (B, Hkv, n), "weights")
    _ints(keep, (B, Hkv, budget), "keep")
    _ints(counts, (B,), "counts")
    lib = load_library()
    with _launch(stream, weights, lens, keep, counts) as s:
        if keep is None:
            keep = weights.new_empty((B, Hkv, max(0, budget)), dtype=torch.int32)
        if counts is None:
            counts = torch.empty_like(lens)
        _check(lib.fmha_evict_select(a, w, n, budget, sinks, recent, keep.data_ptr(), counts.data_ptr(), s))
    return keep, counts


def cache_compact(k, v, keep, counts, dst_start=None, page_table=None, k_out=None, v_out=None, out_page_table=None,
                  weights=None, weights_out=None, stream=None):
    """Moves the kept rows of a cache together: position keep[b, h, i] -> dst_start[b] + i (None: i), i < counts[b].

    keep: int32 [B, Hkv or 1, n] (unit last stride); counts, dst_start: int32 [B]. Without k_out / v_out the rows
    move inside the cache: positions ascend with i, keep[b, h, i] >= dst_start[b] + i, and no page belongs to two
    sequences. With them (and out_page_table when paged) they are copied into another cache, in any order.
    weights fp32 [B, Hkv, n] move along (to weights_out with another cache); entries past the moved ones become 0.
    Returns (k_out, v_out)."""
    if counts is None:
        raise ValueError("counts must be a contiguous int32 tensor")
    tk, tv, B, Hkv, D, capacity, table = _cache_view(k, v, page_table)
    lens = _array(counts, torch.int32, (B,), "counts")
    a = _pack(*_NO_TENSOR, *tk, *tv, *_NO_TENSOR, *_NO_SF, *_NO_SF, B, 0, 0, Hkv, D, capacity, lens, 0, *table, 0.0, 0)
    shape, stride = keep.shape, keep.stride()
    if keep.dtype != torch.int32 or len(shape) != 3 or shape[0] != B or shape[1] not in (1, Hkv) or (
            shape[2] > 1 and stride[2] != 1):
        raise ValueError(f"keep must be int32 [{B}, {Hkv} or 1, n] with unit last stride")
    start = _array(dst_start, torch.int32, (B,), "dst_start")
    if (k_out is None) != (v_out is None) or (k_out is None and (out_page_table is not None or weights_out is not None)):
        raise ValueError("another cache needs k_out and v_out (and, when paged, out_page_table)")
    o = 0
    if k_out is not None:
        if k_out.dtype != k.dtype or v_out.dtype != v.dtype:
            raise ValueError("k_out / v_out must have the dtypes, heads and head dim of k / v")
        ok, ov, out_B, out_Hkv, out_D, room, out_table = _cache_view(k_out, v_out, out_page_table)
        if out_Hkv != Hkv or out_D != D:
            raise ValueError("k_out / v_out must have the dtypes, heads and head dim of k / v")
        if out_B != B:
            raise ValueError(f"caches of {B} and {out_B} sequences")
        o = _pack(*_NO_TENSOR, *ok, *ov, *_NO_TENSOR, *_NO_SF, *_NO_SF, B, 0, 0, Hkv, D, room, lens, 0, *out_table, 0.0, 0)
        if (weights is None) != (weights_out is None):
            raise ValueError("weights and weights_out go together")
    w = wo = nw = nwo = 0
    if weights is not None:
        if weights.dim() != 3 or (weights_out is not None and weights_out.dim() != 3):
            raise ValueError("weights must be contiguous float32 [B, Hkv, n] tensors")
        nw = weights.shape[2]
        w = _array(weights, torch.float32, (B, Hkv, nw), "weights")
        wo, nwo = w, nw
        if weights_out is not None:
            nwo = weights_out.shape[2]
            wo = _array(weights_out, torch.float32, (B, Hkv, nwo), "weights_out")
    _int32s("n", shape[2], nw, nwo)
    lib = load_library()
    with _launch(stream, k, v, keep, counts, dst_start, page_table, k_out, v_out, out_page_table, weights,
                 weights_out) as s:
        _check(lib.fmha_cache_compact(a, o, keep.data_ptr(), stride[0] if B > 1 else 0, stride[1] if shape[1] > 1 else 0,
                                      shape[2], lens, start, w, nw, wo, nwo, s))
    return (k, v) if k_out is None else (k_out, v_out)
