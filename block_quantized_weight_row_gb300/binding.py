"""Thin Python binding over libbq.so (the C ABI in include/bq.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. Tensors must be CUDA tensors; the binding passes their device
pointers, the torch current stream and a torch-allocated workspace to the
library, and raises BQError on a nonzero status. There is no CPU fallback: if
libbq.so is missing or fails to load, every call raises.
"""
import ctypes
import dataclasses
import os
import threading
from typing import NamedTuple

import torch

Q4_0 = 2
Q8_0 = 8
Q4_1, Q5_0, Q5_1 = 3, 6, 7
Q4_K, Q6_K = 12, 14
QK = 32

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libbq.so"

_STATUS = {0: "BQ_OK", -1: "BQ_ERR_INVALID_ARG", -2: "BQ_ERR_SHAPE", -3: "BQ_ERR_UNSUPPORTED",
           -4: "BQ_ERR_ALIGN", -5: "BQ_ERR_CUDA", -6: "BQ_ERR_TIMEOUT", -7: "BQ_ERR_WORKSPACE",
           -8: "BQ_ERR_BASIS", -9: "BQ_ERR_INDEX"}
BASIS_PLAIN, BASIS_HADAMARD64 = 0, 1


ELEM = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class _CacheStruct(ctypes.Structure):
    """bq_paged_cache of include/bq.h"""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("n_kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("k_type", ctypes.c_int), ("v_type", ctypes.c_int), ("k_basis", ctypes.c_int)]


class BQError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


_lib = None


class _Workspaces(threading.local):
    def __init__(self):
        self.stream = None  # of the thread's latest call
        self.eager = {}     # (device, stream) -> uint8 tensor
        self.given = None   # what the library has


_ws = _Workspaces()


def lib():
    """Load libbq.so (built in-tree by build.py); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run __graft_entry__.build() "
                          "(the CUDA path has no fallback)")
    L = ctypes.CDLL(path)
    i, i64, vp, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    cp = ctypes.POINTER(_CacheStruct)
    sig = {
        "bq_quantize_rows": ([i, vp, vp, i64, i64], i),
        "bq_dequantize_rows": ([i, vp, vp, i64, i64], i),
        "bq_gemv": ([i, vp, vp, vp, i64, i64], i),
        "bq_gemv_multi": ([i, i, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(i64), vp, i64], i),
        "bq_gemv_sequence": ([i, i, ctypes.POINTER(i), ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(i64),
                              ctypes.POINTER(vp), ctypes.POINTER(i64)], i),
        "bq_gemv_sequence_workspace_size": ([], sz),
        "bq_attn_decode": ([i, i, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float], i),
        "bq_attn_decode_basis": ([i, i, i, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float], i),
        "bq_kv_quantize_basis": ([i, vp, vp, i, i, vp, i64, i64, i64], i),
        "bq_kv_bias": ([vp, i, vp, i64, i64, i64], i),
        "bq_attn_workspace_size": ([i, i, i64, i64, i64, i64], sz),
        "bq_gemm": ([i, vp, vp, vp, i64, i64, i64], i),
        "bq_kv_quantize": ([i, vp, vp, vp, i64, i64, i64], i),
        "bq_kv_write": ([i, vp, vp, i, i, vp, i, vp, vp, i64, i64, i64], i),
        "bq_paged_page_bytes": ([i, i64, i64, i64], sz),
        "bq_paged_kv_write": ([cp, i, vp, i64, i64, vp, i64, i64, vp, i, vp, i64], i),
        "bq_paged_kv_read": ([cp, i, vp, vp, vp, i, vp, i64], i),
        "bq_paged_attn": ([cp, i, vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                           ctypes.c_float, i, i64], i),
        "bq_paged_attn_workspace_size": ([cp, i, i64, i64, i64, i64, i64, i, i64], sz),
        "bq_paged_attn_many_rows": ([cp, i, i64, i64, i64, i64, i64, i, i64], i64),
        "bq_paged_slot_check": ([cp, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)], i),
        "bq_paged_extend": ([i64, i64, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp], i),
        "bq_add_rms_norm": ([i, vp, i64, vp, i64, vp, ctypes.c_double, vp, i64, vp, i64, vp, i64, i64], i),
        "bq_gemv_q8": ([i, vp, vp, vp, i64, i64], i),
        "bq_gemm_q8": ([i, vp, vp, vp, i64, i64, i64], i),
        "bq_rotary": ([i, vp, i64, i64, i64, vp, i64, i64, i64, i, vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, vp, i64, i64,
                       i64, i, i], i),
        "bq_lora": ([i, vp, i64, i, vp, vp, vp, i64, i64, vp, i, vp, i64, vp, i64, i64, i64, i64], i),
        "bq_lora_workspace_size": ([i64, i64, i64, i64, i64], sz),
        "bq_block_dots": ([i, vp, vp, vp, i64, i64], i),
        "bq_set_stream": ([vp], i),
        "bq_get_stream": ([], vp),
        "bq_set_workspace": ([vp, sz], i),
        "bq_get_workspace": ([ctypes.POINTER(sz)], vp),
        "bq_workspace_size": ([i, i64, i64, i64], sz),
        "bq_gemv_workspace_size": ([i, i64], sz),
        "bq_last_error": ([], ctypes.c_char_p),
        "bq_block_bytes": ([i], i),
        "bq_block_values": ([i], i),
        "bq_device_status": ([], i),
        "bq_version": ([], i),
        "bq_set_spin_limit": ([i64], i),
        "bq_set_weight_prefetch": ([i], i),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
    _lib = L
    return L


def _check(status: int, what: str):
    if status != 0:
        msg = lib().bq_last_error()
        raise BQError(status, f"{what}: {msg.decode() if msg else ''}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _prep(device):
    """Point the library at torch's current stream on `device`."""
    L = lib()
    s = torch.cuda.current_stream(device).cuda_stream
    _check(L.bq_set_stream(s), "bq_set_stream")
    _ws.stream = s
    return L


def clear_workspace() -> None:
    """Detach the calling thread's workspace (GEMVs then quantize x in-kernel)."""
    _check(lib().bq_set_workspace(None, 0), "bq_set_workspace")


def _workspace(device, nbytes: int):
    """Hand the library a torch-owned workspace that nothing else uses meanwhile: a
    thread has one for each stream, which follows its calls there and grows; while a
    graph is captured each call has its own, in the graph's pool, since replays run
    beside later calls of any stream and outlive a growing buffer. (One from the
    allocator for every call costs 5 us of host time.)"""
    capturing = torch.cuda.is_current_stream_capturing()
    key = device, _ws.stream
    ws = None if capturing else _ws.eager.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        if not capturing:
            _ws.eager[key] = ws
    _check(lib().bq_set_workspace(ws.data_ptr(), ws.numel()), "bq_set_workspace")
    _ws.given = ws  # lives as long as the library has its address
    return ws


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _f32(t, name, n=0):
    """A contiguous fp32 tensor of n values at least: the library takes a bare pointer."""
    if _cuda(t, name).dtype != torch.float32:
        raise TypeError(f"{name} must be float32, not {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{name} must have {n} values, not {t.numel()}")
    return t


def _rows(x, name, rows, K):
    """Activations: fp32 values, or whole rows as Q8_0 blocks (the bytes)."""
    if x.dtype != torch.uint8:
        return _f32(x, name, rows * K)
    n = rows * (K // QK) * 34
    if _cuda(x, name).numel() != n:
        raise ValueError(f"{name}: {rows} x {K} values in Q8_0 are {n} bytes, not {x.numel()}")
    return x


def block_bytes(t: int) -> int:
    return int(lib().bq_block_bytes(t))


def block_values(t: int) -> int:
    return int(lib().bq_block_values(t))


def quantize_rows(t: int, src: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp32 (rows, cols) -> uint8 (rows, cols/32*block_bytes)."""
    _cuda(src, "src")
    if src.dtype != torch.float32:
        raise TypeError("src must be float32")
    x = src.reshape(-1, src.shape[-1]) if src.dim() != 2 else src
    R, C = x.shape
    if out is None:
        out = torch.empty((R, (C // max(block_values(t), 1)) * max(block_bytes(t), 1)), dtype=torch.uint8,
                          device=src.device)
    L = _prep(src.device)
    _check(L.bq_quantize_rows(t, _ptr(x), _ptr(out), R, C), "bq_quantize_rows")
    return out


def dequantize_rows(t: int, blocks: torch.Tensor, cols: int, out: torch.Tensor | None = None) -> torch.Tensor:
    _cuda(blocks, "blocks")
    nbr = (cols // max(block_values(t), 1)) * block_bytes(t)
    R = blocks.numel() // nbr if nbr else 0
    try:
        ext = _ext or _paged()
    except ImportError:  # the library alone serves this call too, with more host time
        return _dequantize_rows(t, blocks, R, cols, out)
    r = ext.dequantize_rows(t, blocks, R, cols, out)
    if type(r) is tuple:
        _raise(r, "bq_dequantize_rows")
    return r


def _dequantize_rows(t, blocks, R, cols, out):
    if blocks.dtype != torch.uint8:
        raise TypeError(f"blocks must be uint8, not {blocks.dtype}")
    if out is None:
        out = torch.empty((R, cols), dtype=torch.float32, device=blocks.device)
    elif _f32(out, "out", R * cols).device != blocks.device:
        raise ValueError("out is on another device than blocks")
    with torch.cuda.device(blocks.device):
        L = _prep(blocks.device)
        _check(L.bq_dequantize_rows(t, _ptr(blocks), _ptr(out), R, cols), "bq_dequantize_rows")
    return out


def gemv(t: int, w_blocks: torch.Tensor, x: torch.Tensor, M: int, K: int,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """y[M] = W (M x K, blocks of type t) . x[K] (fp32, quantized to Q8_0 in-kernel;
    or uint8: its Q8_0 blocks, as add_rms_norm and quantize_rows give them)."""
    _cuda(w_blocks, "w_blocks")
    _rows(x, "x", 1, K)
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=x.device)
    else:
        _f32(out, "out", M)
    L = _prep(x.device)
    _workspace(x.device, int(L.bq_gemv_workspace_size(t, K)))
    if x.dtype == torch.uint8:
        _check(L.bq_gemv_q8(t, _ptr(w_blocks), _ptr(x), _ptr(out), M, K), "bq_gemv_q8")
        return out
    _check(L.bq_gemv(t, _ptr(w_blocks), _ptr(x), _ptr(out), M, K), "bq_gemv")
    return out


def gemv_multi_args(w_list, y_list, M_list):
    """ctypes arrays (W pointers, y pointers, row counts) for bq_gemv_multi."""
    n = len(w_list)
    W = (ctypes.c_void_p * n)(*[w.data_ptr() for w in w_list])
    Y = (ctypes.c_void_p * n)(*[y.data_ptr() for y in y_list])
    M = (ctypes.c_int64 * n)(*M_list)
    return n, W, Y, M


def gemv_multi(t: int, w_list, x: torch.Tensor, M_list, K: int, outs=None):
    """y_i = W_i . x for matrices sharing one input x, in one launch."""
    for w in w_list:
        _cuda(w, "w_blocks")
    _f32(x, "x", K)
    if outs is None:
        outs = [torch.empty(m, dtype=torch.float32, device=x.device) for m in M_list]
    else:
        for y, m in zip(outs, M_list):
            _f32(y, "outs", m)
    n, W, Y, M = gemv_multi_args(w_list, outs, M_list)
    L = _prep(x.device)
    _workspace(x.device, int(L.bq_gemv_workspace_size(t, K)))
    _check(L.bq_gemv_multi(t, n, W, Y, M, _ptr(x), K), "bq_gemv_multi")
    return outs


def gemv_sequence_args(groups):
    """ctypes arrays for bq_gemv_sequence from batches (w_list, x, M_list, K, outs).
    Building them once and passing them to gemv_sequence_call keeps the
    per-call host work to one C call."""
    n_groups = len(groups)
    n_mats = (ctypes.c_int * n_groups)(*[len(g[0]) for g in groups])
    ws = [w for g in groups for w in g[0]]
    ys = [y for g in groups for y in g[4]]
    ms = [m for g in groups for m in g[2]]
    W = (ctypes.c_void_p * len(ws))(*[w.data_ptr() for w in ws])
    Y = (ctypes.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
    M = (ctypes.c_int64 * len(ms))(*ms)
    X = (ctypes.c_void_p * n_groups)(*[g[1].data_ptr() for g in groups])
    K = (ctypes.c_int64 * n_groups)(*[g[3] for g in groups])
    return (n_groups, n_mats, W, Y, M, X, K)


def gemv_sequence_call(t: int, args, device):
    L = _prep(device)
    _workspace(device, int(L.bq_gemv_sequence_workspace_size()))
    _check(L.bq_gemv_sequence(t, *args), "bq_gemv_sequence")


def gemv_sequence(t: int, groups):
    """Batches (w_list, x, M_list, K, outs) in one launch; batch g reads its x
    after the outputs of batches 0..g-1 are written. outs may be None."""
    full = []
    for w_list, x, M_list, K, outs in groups:
        for w in w_list:
            _cuda(w, "w_blocks")
        _f32(x, "x", K)
        if outs is None:
            outs = [torch.empty(m, dtype=torch.float32, device=x.device) for m in M_list]
        else:
            for y, m in zip(outs, M_list):
                _f32(y, "outs", m)
        full.append((w_list, x, M_list, K, outs))
    if full:
        gemv_sequence_call(t, gemv_sequence_args(full), full[0][1].device)
    return [g[4] for g in full]


def attn_decode(k_type: int, v_type: int, q: torch.Tensor, K_cache: torch.Tensor, V_cache: torch.Tensor,
                n_kv_heads: int, scale: float, out: torch.Tensor | None = None,
                k_basis: int = BASIS_PLAIN) -> torch.Tensor:
    """o (n_heads, head_dim) = attention of q (n_heads, head_dim) over the
    quantized caches (n_tokens, n_kv_heads, head_dim/32 blocks as bytes);
    k_basis: the basis the K cache was written in."""
    _f32(q, "q")
    _cuda(K_cache, "K_cache")
    _cuda(V_cache, "V_cache")
    H, D = q.shape
    T = K_cache.shape[0]
    if out is None:
        out = torch.empty((H, D), dtype=torch.float32, device=q.device)
    L = _prep(q.device)
    _workspace(q.device, int(L.bq_attn_workspace_size(k_type, v_type, T, H, n_kv_heads, D)))
    _check(L.bq_attn_decode_basis(k_type, v_type, k_basis, _ptr(q), _ptr(K_cache), _ptr(V_cache), _ptr(out), T, H,
                                  n_kv_heads, D, float(scale)), "bq_attn_decode_basis")
    return out


def gemm(t: int, w_blocks: torch.Tensor, X: torch.Tensor, M: int, N: int, K: int,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """Y (N x M) = X (N x K fp32, quantized to Q8_0; or uint8: its Q8_0 blocks) . W^T
    (W: M x K blocks)."""
    _cuda(w_blocks, "w_blocks")
    _rows(X, "X", N, K)
    if out is None:
        out = torch.empty((N, M), dtype=torch.float32, device=X.device)
    else:
        _f32(out, "out", N * M)
    L = _prep(X.device)
    _workspace(X.device, int(L.bq_workspace_size(t, M, N, K)))
    if X.dtype == torch.uint8:
        _check(L.bq_gemm_q8(t, _ptr(w_blocks), _ptr(X), _ptr(out), M, N, K), "bq_gemm_q8")
        return out
    _check(L.bq_gemm(t, _ptr(w_blocks), _ptr(X), _ptr(out), M, N, K), "bq_gemm")
    return out


def kv_quantize(t: int, rows: torch.Tensor, bias: torch.Tensor | None,
                out: torch.Tensor | None = None, basis: int = BASIS_PLAIN,
                bias_basis: int | None = None) -> torch.Tensor:
    """rows: (n_tokens, n_kv_heads, head_dim) fp32; bias: (n_kv_heads, head_dim) or None.
    basis: the cache's basis; bias_basis: the basis the bias was calibrated in
    (default: the cache's)."""
    _f32(rows, "rows")
    if bias is not None:
        _f32(bias, "bias")
    T, H, D = rows.shape
    if out is None:
        out = torch.empty((T, H, (D // QK) * max(block_bytes(t), 1)), dtype=torch.uint8, device=rows.device)
    L = _prep(rows.device)
    _check(L.bq_kv_quantize_basis(t, _ptr(rows), _ptr(bias), basis if bias_basis is None else bias_basis, basis,
                                  _ptr(out), T, H, D), "bq_kv_quantize_basis")
    return out


def kv_write(k_type: int, k_rows: torch.Tensor, bias: torch.Tensor | None, v_type: int, v_rows: torch.Tensor,
             out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None, basis: int = BASIS_PLAIN,
             bias_basis: int | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """One layer's K and V cache write in one launch (bq_kv_write): k_rows and
    v_rows (n_tokens, n_kv_heads, head_dim) fp32; bias (n_kv_heads, head_dim)
    or None; basis: the K cache's basis. Returns (K blocks, V blocks)."""
    _f32(k_rows, "k_rows")
    _f32(v_rows, "v_rows")
    if bias is not None:
        _f32(bias, "bias")
    T, H, D = k_rows.shape
    if tuple(v_rows.shape) != (T, H, D):
        raise ValueError("k_rows and v_rows must have the same shape")
    if out_k is None:
        out_k = torch.empty((T, H, (D // QK) * max(block_bytes(k_type), 1)), dtype=torch.uint8, device=k_rows.device)
    if out_v is None:
        out_v = torch.empty((T, H, (D // QK) * max(block_bytes(v_type), 1)), dtype=torch.uint8, device=v_rows.device)
    L = _prep(k_rows.device)
    _check(L.bq_kv_write(k_type, _ptr(k_rows), _ptr(bias), basis if bias_basis is None else bias_basis, basis,
                         _ptr(out_k), v_type, _ptr(v_rows), _ptr(out_v), T, H, D), "bq_kv_write")
    return out_k, out_v


def kv_bias(rows: torch.Tensor, basis: int = BASIS_PLAIN, out: torch.Tensor | None = None) -> torch.Tensor:
    """Mean-centering bias (n_kv_heads, head_dim) fp32 of calibration rows
    (n_tokens, n_kv_heads, head_dim), measured in `basis`."""
    _f32(rows, "rows")
    T, H, D = rows.shape
    if out is None:
        out = torch.empty((H, D), dtype=torch.float32, device=rows.device)
    L = _prep(rows.device)
    _check(L.bq_kv_bias(_ptr(rows), basis, _ptr(out), T, H, D), "bq_kv_bias")
    return out


# ---- paged KV cache ----
# The tensors are checked and the library called in _paged.so (csrc/paged_binding.cpp).

_ext = None


def _paged():
    """Load _paged.so (built in-tree by build.py); raise if it is missing."""
    global _ext
    if _ext is None:
        lib()
        try:
            from . import _paged as ext
        except ImportError as e:
            raise ImportError(f"the paged calls' _paged.so is not built or does not load ({e}); run "
                              "__graft_entry__.build() (the CUDA path has no fallback)") from e
        _ext = ext
    return _ext


@dataclasses.dataclass
class PagedCache:
    """One layer's paged KV cache: two pools of pages (layout in include/bq.h),
    each uint8 (n_pages, n_kv_heads, page_size * head_dim / 32 * block bytes)."""
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    page_size: int
    head_dim: int
    k_type: int = Q4_0
    v_type: int = Q4_0
    k_basis: int = BASIS_PLAIN

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, k_type: int = Q4_0,
              v_type: int = Q4_0, k_basis: int = BASIS_PLAIN, device="cuda") -> "PagedCache":
        """A cache of n_pages pages of unwritten content."""
        pools = []
        for t in (k_type, v_type):
            n = int(lib().bq_paged_page_bytes(t, page_size, n_kv_heads, head_dim))
            if n == 0:
                raise BQError(-2, f"no page of type {t} has page_size {page_size}, {n_kv_heads} heads, head_dim {head_dim}")
            pools.append(torch.empty((n_pages, n_kv_heads, n // n_kv_heads), dtype=torch.uint8, device=device))
        return cls(pools[0], pools[1], page_size, head_dim, k_type, v_type, k_basis)


def paged_kv_write(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                   bias: torch.Tensor | None = None, bias_basis: int | None = None) -> None:
    """Quantize the rows k and v (tokens, n_kv_heads, head_dim; fp32, fp16 or
    bf16, any token and head strides) into the cache at slots (int64, page *
    page_size + place; -1 skips a token). bias (n_kv_heads, head_dim) fp32:
    subtracted from K, calibrated in bias_basis (default: the cache's)."""
    r = (_ext or _paged()).kv_write(cache.k_pages, cache.v_pages, cache.page_size, cache.head_dim, cache.k_type,
                                    cache.v_type, cache.k_basis, k, v, slots, bias, bias_basis)
    if r is not None:
        _check(r, "bq_paged_kv_write")


def paged_kv_read(cache: PagedCache, slots: torch.Tensor, dtype: torch.dtype = torch.float32,
                  bias: torch.Tensor | None = None, bias_basis: int | None = None,
                  out_k: torch.Tensor | None = None,
                  out_v: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """The rows at slots (int64; -1: zeros) as (K, V), each (tokens,
    n_kv_heads, head_dim) of dtype; K out of the cache's basis, plus bias."""
    r = (_ext or _paged()).kv_read(cache.k_pages, cache.v_pages, cache.page_size, cache.head_dim, cache.k_type,
                                   cache.v_type, cache.k_basis, slots, ELEM.get(dtype, -1), bias, bias_basis,
                                   out_k, out_v)
    if type(r) is int:
        _check(r, "bq_paged_kv_read")
    return r


def paged_attn(cache: PagedCache, q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
               page_table: torch.Tensor, scale: float, *, max_q_len: int, max_kv_len: int, causal: bool = True,
               window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of a batch of sequences over the cache (bq_paged_attn): q
    (tokens, n_heads, head_dim), sequence b's tokens q_start[b] .. q_start[b +
    1] - 1 being the last of its kv_len[b] cached ones; page_table (sequences,
    max_pages). The index tensors are int32 on the device; max_q_len and
    max_kv_len are their bounds on the host. window: tokens a causal query
    sees (0: all). lse: optional fp32 (tokens, n_heads), written."""
    r = (_ext or _paged()).attn(cache.k_pages, cache.v_pages, cache.page_size, cache.head_dim, cache.k_type,
                                cache.v_type, cache.k_basis, q, q_start, kv_len, page_table, scale, max_q_len,
                                max_kv_len, causal, window, out, lse)
    if type(r) is tuple:
        raise BQError(r[0], f"bq_paged_attn: {r[1]}")
    return r


# ---- around the projections and the paged cache of a served layer ----


def _raise(r, what):
    raise BQError(r[0], f"{what}: {r[1]}")


class PagedStep(NamedTuple):
    """What paged_extend makes of a batch's lengths (all on the device). The tensors lie
    in one allocation, which each of them keeps alive: copy what outlives the step."""
    q_start: torch.Tensor    # int32 (sequences + 1): rows of each sequence in the batch
    kv_len: torch.Tensor     # int32 (sequences): tokens cached once the step's rows are written
    slots: torch.Tensor      # int64 (n_slots): where each row goes, -1 behind the last
    positions: torch.Tensor  # int32 (n_slots): each row's place in its sequence, 0 behind the last
    taken: torch.Tensor      # int32 (2): pages taken off the front of free_pages; pages needed


def paged_extend(page_size: int, n_pages: int, kv_len: torch.Tensor, n_new: torch.Tensor, page_table: torch.Tensor,
                 free_pages: torch.Tensor, n_slots: int) -> PagedStep:
    """The next tokens of a batch of sequences in paged caches of n_pages pages
    (bq_paged_extend): kv_len and n_new (sequences) int32, the cached and the coming
    tokens; page_table (sequences, max_pages) int32, to which new pages are added in
    place, from the front of free_pages (int32), which the caller moves on by taken[0]
    before the next call; n_slots: room for the batch's tokens. A sequence that cannot grow gets slots of -1 and keeps its kv_len, which
    device_status reports; taken[1] > taken[0] tells so too where pages ran out."""
    r = (_ext or _paged()).paged_extend(page_size, n_pages, kv_len, n_new, page_table, free_pages, n_slots)
    if type(r[0]) is int:
        _raise(r, "bq_paged_extend")
    return PagedStep(*r)


class NormRows(NamedTuple):
    """Outputs of add_rms_norm; None where not wanted."""
    out: torch.Tensor | None  # the norm's rows, in x's type
    sum: torch.Tensor | None  # x + residual, in x's type
    q8: torch.Tensor | None   # the norm's rows in Q8_0: uint8 (rows, cols / 32 * 34)


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None, *,
                 out: bool | torch.Tensor = True, q8: bool | torch.Tensor = False,
                 sum: torch.Tensor | None = None) -> NormRows:
    """Root-mean-square norm of the rows x + residual (bq_add_rms_norm): x and
    residual (rows, cols) fp32, fp16 or bf16, any row stride; weight (cols) fp32. out
    and q8: which of the two outputs to make, or a tensor for it; sum: a tensor for
    x + residual (x or residual themselves: in place), else a new one is made."""
    r = (_ext or _paged()).add_rms_norm(x, weight, eps, residual, out, q8, sum)
    if type(r[0]) is int:
        _raise(r, "bq_add_rms_norm")
    return NormRows(*r)


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
           axis: torch.Tensor | None = None, *, interleaved: bool = False, inverse: bool = False,
           dtype: torch.dtype | None = None, out_q: torch.Tensor | None = None,
           out_k: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Rotary positions (bq_rotary): q and k (tokens, heads, head_dim), any token and
    head strides, turned in their first 2 * len(inv_freq) channels by positions (int32,
    (axes, tokens) or (tokens)) of the axis of each pair (axis: int32, None: the first)
    times inv_freq (fp64). interleaved: pairs of adjacent channels, else of the two
    halves. inverse: the opposite turn. dtype: of the outputs (from fp32 any; else q's).
    out_q, out_k may be q and k themselves."""
    code = -1 if dtype is None else ELEM.get(dtype, 3)
    if dtype is None and out_q is not None:
        code = ELEM.get(out_q.dtype, 3)
    r = (_ext or _paged()).rotary(q, k, positions, inv_freq, axis, interleaved, inverse, code, out_q, out_k)
    if type(r[0]) is int:
        _raise(r, "bq_rotary")
    return r


def lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapter: torch.Tensor, y: torch.Tensor | None = None,
         scale: torch.Tensor | None = None, *, out: torch.Tensor | None = None,
         dtype: torch.dtype | None = None) -> torch.Tensor:
    """y + scale[adapter] * (x a[adapter]^T) b[adapter]^T per row (bq_lora): x (tokens,
    K) and y (tokens, M) fp32 or in the adapters' type; a (adapters, rank, K) and b
    (adapters, M, rank) fp16 or bf16; adapter (tokens) int32, -1 for none; scale
    (adapters) fp32, None for 1. out may be y itself. Without y, nothing is added to,
    and dtype is out's (default: x's)."""
    code = -1 if dtype is None else ELEM.get(dtype, 3)
    r = (_ext or _paged()).lora(x, a, b, adapter, y, scale, out, code)
    if type(r) is tuple:
        _raise(r, "bq_lora")
    return r


def block_dots(t: int, w_blocks: torch.Tensor, xq_blocks: torch.Tensor, M: int, K: int) -> torch.Tensor:
    """Test export: int32 (M, K/32) per-block integer dots of W against Q8_0 blocks xq."""
    _cuda(w_blocks, "w_blocks")
    _cuda(xq_blocks, "xq_blocks")
    out = torch.empty((M, K // QK), dtype=torch.int32, device=w_blocks.device)
    L = _prep(w_blocks.device)
    _check(L.bq_block_dots(t, _ptr(w_blocks), _ptr(xq_blocks), _ptr(out), M, K), "bq_block_dots")
    return out


def set_weight_prefetch(enable: bool) -> None:
    """Let the calling thread's GEMVs stream weights before the previous
    kernel on the stream has completed (only for weights no running kernel
    writes)."""
    _check(lib().bq_set_weight_prefetch(1 if enable else 0), "bq_set_weight_prefetch")


def device_status() -> int:
    """Synchronize the current stream and return (and clear) the device error word."""
    return int(lib().bq_device_status())
