"""ctypes binding of libattn_b200.so: argument marshalling only.

Each function here has the name of a C entry point of include/attn_b200.h.  It checks
that torch tensors have the dtype, device and layout the C side expects, reads their
sizes and device addresses, and calls the C function on the given (default: current)
CUDA stream.  All computation happens in the library's kernels.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None
_LOCK = threading.Lock()

ATTN_OK = 0
STATUS_NAMES = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_ALIGNMENT",
                4: "ATTN_ERR_CUDA", 5: "ATTN_ERR_DEVICE_TIMEOUT", 6: "ATTN_ERR_BAD_PAGE",
                7: "ATTN_ERR_WORKSPACE", 8: "ATTN_ERR_TOO_LARGE"}
DTYPE_BF16, DTYPE_F32 = 0, 1

# exported symbol -> (restype, argtypes); mirrors include/attn_b200.h
_P = ctypes.c_void_p
_I = ctypes.c_int
SIGNATURES = {
    "attn_abi_version": (_I, []),
    "attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I, _P]),
    "attn_fwd_ex": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I, _P]),
    "attn_fwd_masked": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I, _I, _P, _P]),
    "attn_quantize_fp8": (_I, [_P, _P, _P, _I, _I, _I, _I, _P]),
    "attn_fwd_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I, _P]),
    "attn_bwd_workspace_size": (ctypes.c_size_t, [_I, _I, _I]),
    "attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I, _P,
                      ctypes.c_size_t, _P]),
    "attn_decode_paged_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "attn_decode_paged": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P,
                               ctypes.c_size_t, _P]),
    "attn_decode_paged_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float,
                                       _P]),
    "attn_decode_paged_noalloc_max_scratch": (ctypes.c_size_t, []),
    "attn_kv4_page_bytes": (ctypes.c_size_t, [_I, _I, _I]),
    "attn_kv4_append": (_I, [_P, _P, ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                             _I, _P]),
    "attn_kv4_gather": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "attn_decode_paged_kv4_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "attn_decode_paged_kv4": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P,
                                   ctypes.c_size_t, _P]),
    "attn_pages_workspace_size": (ctypes.c_size_t, [_I, _I]),
    "attn_pages_fork": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, ctypes.c_size_t, _I, _I, _I, _I, _I, _P, _P,
                             ctypes.c_size_t, _P]),
    "attn_pages_compact": (_I, [_P, _P, _P, _P, _I, _P, _I, ctypes.c_size_t, _I, _I, _I, _P, _P, ctypes.c_size_t,
                                _P]),
    "attn_debug_watchdog": (_I, [ctypes.c_uint64, _P]),
    "attn_debug_exp2": (_I, [_P, _P, _I, _P]),
    "attn_debug_fwd_stall": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I, _I, _I,
                                  ctypes.c_uint64, _P]),
    "attn_debug_bwd_stall": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I,
                                  _P, ctypes.c_size_t, _I, _I, ctypes.c_uint64, _P]),
    "attn_debug_decode_stall": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P,
                                     ctypes.c_size_t, _I, _I, ctypes.c_uint64, _P]),
    "attn_get_device_status": (_I, [_P]),
    "attn_status_string": (ctypes.c_char_p, [_I]),
}


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


def library_path() -> str:
    return os.path.join(_HERE, "libattn_b200.so")


def load_library() -> ctypes.CDLL:
    """Loads the CUDA library; raises RuntimeError if it is missing or cannot be loaded."""
    global _LIB
    with _LOCK:
        if _LIB is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is not built: run `python -m attn_fwd_05_b200.build`")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _LIB = lib
    return _LIB


def _stream(stream) -> int | None:
    if stream is None:
        # the handle alone where this PyTorch gives it: building a torch.cuda.Stream costs 3 us a call
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str) -> None:
    if status != ATTN_OK:
        raise AttnError(status, where)


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int | None = None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    return t.data_ptr()


def _fwd_shapes(q, k, v, o, lse):
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Hkv, Nk, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, Hkv, Nk, d] with q's B and d")
    if tuple(o.shape) != (B, Hq, Nq, d):
        raise ValueError("o must be [B, Hq, Nq, d]")
    if lse is not None and tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("lse must be [B, Hq, Nq]")
    if o.dtype == torch.bfloat16:
        odt = DTYPE_BF16
    elif o.dtype == torch.float32:
        odt = DTYPE_F32
    else:
        raise TypeError("o must be bf16 or fp32")
    ptrs = (_dev(q, "q", torch.bfloat16, 4), _dev(k, "k", torch.bfloat16, 4), _dev(v, "v", torch.bfloat16, 4),
            _dev(o, "o", o.dtype, 4), odt, None if lse is None else _dev(lse, "lse", torch.float32, 3))
    return ptrs, (B, Hq, Hkv, Nq, Nk, d)


def attn_fwd_ex(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor | None,
                causal: bool, scale: float, stream=None) -> None:
    """Prefill forward; o is bf16 or fp32 [B, Hq, Nq, d], lse fp32 [B, Hq, Nq] or None."""
    lib = load_library()
    ptrs, dims = _fwd_shapes(q, k, v, o, lse)
    st = lib.attn_fwd_ex(*ptrs, *dims, float(scale), int(bool(causal)), _stream(stream))
    _check(st, "attn_fwd_ex")


def attn_fwd_masked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor | None,
                    causal: bool, scale: float, window: int = 0, block_mask: torch.Tensor | None = None,
                    stream=None) -> None:
    """Prefill forward with a sliding window (window > 0, needs causal) and/or a
    block-sparse map: uint8 [ceil(Nq/128), ceil(Nk/128)] on the device, nonzero =
    the 128 x 128 block pair attends."""
    lib = load_library()
    ptrs, dims = _fwd_shapes(q, k, v, o, lse)
    bm = None
    if block_mask is not None:
        Nq, Nk = dims[3], dims[4]
        want = ((Nq + 127) // 128, (Nk + 127) // 128)
        if tuple(block_mask.shape) != want:
            raise ValueError(f"block_mask must be {want}")
        bm = _dev(block_mask, "block_mask", torch.uint8, 2)
    st = lib.attn_fwd_masked(*ptrs, *dims, float(scale), int(bool(causal)), int(window), bm, _stream(stream))
    _check(st, "attn_fwd_masked")


def attn_fwd(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    """Prefill forward with bf16 output (see attn_fwd_ex)."""
    if o.dtype != torch.bfloat16:
        raise TypeError("attn_fwd writes bf16 o; use attn_fwd_ex for fp32")
    attn_fwd_ex(q, k, v, o, lse, causal, scale, stream)


def attn_quantize_fp8(x: torch.Tensor, block_rows: int, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Block e4m3 quantization of a bf16 [..., N, d] tensor: returns (codes uint8 [..., N, d],
    scales fp32 [..., ceil(N / block_rows)])."""
    lib = load_library()
    *lead, N, d = x.shape
    planes = 1
    for n in lead:
        planes *= n
    nblk = (N + block_rows - 1) // block_rows
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty((*lead, nblk), dtype=torch.float32, device=x.device)
    st = lib.attn_quantize_fp8(_dev(x, "x", torch.bfloat16), out.data_ptr(), scales.data_ptr(), planes, N, d,
                               block_rows, _stream(stream))
    _check(st, "attn_quantize_fp8")
    return out, scales


def attn_fwd_fp8(q8, q_scale, k8, k_scale, v8, v_scale, o, lse, causal: bool, scale: float, stream=None) -> None:
    """FP8 forward: e4m3 q8 [B, Hq, Nq, 128], k8/v8 [B, Hkv, Nk, 128] (uint8 tensors) with fp32
    scales q_scale [B, Hq, ceil(Nq/128)], k_scale [B, Hkv, ceil(Nk/128)], v_scale [B, Hkv]."""
    lib = load_library()
    B, Hq, Nq, d = q8.shape
    Hkv, Nk = k8.shape[1], k8.shape[2]
    if tuple(k8.shape) != (B, Hkv, Nk, d) or tuple(v8.shape) != tuple(k8.shape):
        raise ValueError("k8 and v8 must be [B, Hkv, Nk, d]")
    if tuple(q_scale.shape) != (B, Hq, (Nq + 127) // 128) or tuple(k_scale.shape) != (B, Hkv, (Nk + 127) // 128) \
            or tuple(v_scale.shape) != (B, Hkv):
        raise ValueError("scale shapes must be [B, Hq, ceil(Nq/128)], [B, Hkv, ceil(Nk/128)], [B, Hkv]")
    if tuple(o.shape) != (B, Hq, Nq, d):
        raise ValueError("o must be [B, Hq, Nq, d]")
    odt = DTYPE_BF16 if o.dtype == torch.bfloat16 else DTYPE_F32 if o.dtype == torch.float32 else None
    if odt is None:
        raise TypeError("o must be bf16 or fp32")
    st = lib.attn_fwd_fp8(_dev(q8, "q8", torch.uint8, 4), _dev(q_scale, "q_scale", torch.float32, 3),
                          _dev(k8, "k8", torch.uint8, 4), _dev(k_scale, "k_scale", torch.float32, 3),
                          _dev(v8, "v8", torch.uint8, 4), _dev(v_scale, "v_scale", torch.float32, 2),
                          _dev(o, "o", o.dtype, 4), odt, None if lse is None else _dev(lse, "lse", torch.float32, 3),
                          B, Hq, Hkv, Nq, Nk, d, float(scale), int(bool(causal)), _stream(stream))
    _check(st, "attn_fwd_fp8")


def attn_bwd_workspace_size(B: int, Hq: int, Nq: int) -> int:
    return int(load_library().attn_bwd_workspace_size(B, Hq, Nq))


def _bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, scale, workspace):
    lib = load_library()
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Hkv, Nk, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, Hkv, Nk, d] with q's B and d")
    for name, t in (("o", o), ("do", do), ("dq", dq)):
        if tuple(t.shape) != (B, Hq, Nq, d):
            raise ValueError(f"{name} must be [B, Hq, Nq, d]")
    for name, t in (("dk", dk), ("dv", dv)):
        if tuple(t.shape) != (B, Hkv, Nk, d):
            raise ValueError(f"{name} must be [B, Hkv, Nk, d]")
    if tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("lse must be [B, Hq, Nq]")
    need = lib.attn_bwd_workspace_size(B, Hq, Nq)
    if workspace is None:
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=q.device)
    return (_dev(q, "q", torch.bfloat16, 4), _dev(k, "k", torch.bfloat16, 4), _dev(v, "v", torch.bfloat16, 4),
            _dev(o, "o", torch.bfloat16, 4), _dev(do, "do", torch.bfloat16, 4),
            _dev(lse, "lse", torch.float32, 3), _dev(dq, "dq", torch.float32, 4),
            _dev(dk, "dk", torch.float32, 4), _dev(dv, "dv", torch.float32, 4),
            B, Hq, Hkv, Nq, Nk, d, float(scale), int(bool(causal)),
            _dev(workspace, "workspace", torch.uint8, 1), workspace.numel())


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, do: torch.Tensor,
             lse: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, causal: bool, scale: float,
             workspace: torch.Tensor | None = None, stream=None) -> None:
    """Backward pass: fp32 dq [B, Hq, Nq, d], dk and dv [B, Hkv, Nk, d] from the bf16 inputs, the
    forward's bf16 o and fp32 lse, and the bf16 upstream gradient do [B, Hq, Nq, d]."""
    args = _bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, scale, workspace)
    _check(load_library().attn_bwd(*args, _stream(stream)), "attn_bwd")


def attn_decode_paged_workspace_size(num_seqs: int, Hq: int, Hkv: int, d: int, max_pages_per_seq: int,
                                     page_size: int) -> int:
    return int(load_library().attn_decode_paged_workspace_size(num_seqs, Hq, Hkv, d, max_pages_per_seq,
                                                               page_size))


def attn_decode_paged(q, k_pool, v_pool, block_table, seq_lens, page_size: int, o, lse, scale: float,
                      workspace: torch.Tensor, stream=None) -> None:
    """One decode step over a paged KV cache (shapes as in include/attn_b200.h)."""
    lib = load_library()
    S, Hq, d = q.shape
    num_pages, Hkv, ps, d2 = k_pool.shape
    if ps != page_size or d2 != d or tuple(v_pool.shape) != tuple(k_pool.shape):
        raise ValueError("pools must be [num_pages, Hkv, page_size, d]")
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError("block_table must be [num_seqs, max_pages_per_seq]")
    max_pages = block_table.shape[1]
    st = lib.attn_decode_paged(
        _dev(q, "q", torch.bfloat16, 3), _dev(k_pool, "k_pool", torch.bfloat16, 4),
        _dev(v_pool, "v_pool", torch.bfloat16, 4), _dev(block_table, "block_table", torch.int32, 2),
        _dev(seq_lens, "seq_lens", torch.int32, 1), page_size, _dev(o, "o", torch.bfloat16, 3),
        None if lse is None else _dev(lse, "lse", torch.float32, 2), S, Hq, Hkv, d, num_pages, max_pages,
        float(scale), _dev(workspace, "workspace", workspace.dtype), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "attn_decode_paged")


def attn_decode_paged_noalloc(q, k_pool, v_pool, block_table, seq_lens, page_size: int, o, lse, scale: float,
                              stream=None) -> None:
    """attn_decode_paged without a workspace: the library's static scratch is used.

    For callers that must not allocate device memory; raises AttnError with
    ATTN_ERR_TOO_LARGE when the sizes need more scratch than the library holds.
    """
    lib = load_library()
    S, Hq, d = q.shape
    num_pages, Hkv, ps, d2 = k_pool.shape
    if ps != page_size or d2 != d or tuple(v_pool.shape) != tuple(k_pool.shape):
        raise ValueError("pools must be [num_pages, Hkv, page_size, d]")
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError("block_table must be [num_seqs, max_pages_per_seq]")
    st = lib.attn_decode_paged_noalloc(
        _dev(q, "q", torch.bfloat16, 3), _dev(k_pool, "k_pool", torch.bfloat16, 4),
        _dev(v_pool, "v_pool", torch.bfloat16, 4), _dev(block_table, "block_table", torch.int32, 2),
        _dev(seq_lens, "seq_lens", torch.int32, 1), page_size, _dev(o, "o", torch.bfloat16, 3),
        None if lse is None else _dev(lse, "lse", torch.float32, 2), S, Hq, Hkv, d, num_pages,
        block_table.shape[1], float(scale), _stream(stream))
    _check(st, "attn_decode_paged_noalloc")


def _current_device() -> int:
    """Number of the current CUDA device; one that no tensor has where there is no device."""
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2


def _ptr(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int, dev: int) -> int:
    """Address of a dense tensor on device `dev` (the current one, where the call's kernels run)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.dim() == ndim:
        return t.data_ptr()
    _dev(t, name, dtype, ndim)  # says what is wrong, unless it is the device
    raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")


def _scratch(workspace: torch.Tensor, dev: int) -> tuple[int, int]:
    """Address and bytes of a workspace (any type and shape)."""
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    return _ptr(workspace, "workspace", workspace.dtype, workspace.dim(), dev), workspace.nbytes


def _kv4_pool(kv_pool, block_table, seq_lens, page_size: int, d: int, dev: int) -> tuple:
    """Checks a 4-bit pool and its table: ((pool, table, lens) addresses, S, Hkv, num_pages, max_pages)."""
    ptrs = (_ptr(kv_pool, "kv_pool", torch.uint8, 3, dev), _ptr(block_table, "block_table", torch.int32, 2, dev),
            _ptr(seq_lens, "seq_lens", torch.int32, 1, dev))
    S, max_pages = block_table.shape
    if seq_lens.shape[0] != S:
        raise ValueError("seq_lens must be [num_seqs] with block_table's num_seqs")
    num_pages, Hkv, head_bytes = kv_pool.shape
    if head_bytes * 8 != page_size * d * 9:
        raise ValueError(f"kv_pool must be [num_pages, Hkv, page_size * d * 9 / 8] = [.., .., {page_size * d * 9 // 8}]")
    return ptrs, S, Hkv, num_pages, max_pages


def attn_kv4_page_bytes(Hkv: int, page_size: int, d: int) -> int:
    """Bytes of one page of a 4-bit pool; the pool is uint8 [num_pages, Hkv, page_size * d * 9 / 8]."""
    return int(load_library().attn_kv4_page_bytes(Hkv, page_size, d))


def _token_rows(t, name: str, shape, dev: int) -> tuple[int, int]:
    """Address and token stride of a bf16 [T, Hkv, d] tensor whose tokens are dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on a CUDA device, the current one")
    if t.shape != shape:
        raise ValueError(f"{name} must be [num_new, Hkv, d]")
    T, Hkv, d = shape
    st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (Hkv > 1 and sh != d):
        raise ValueError(f"the heads and channels of a token of {name} must be dense")
    return t.data_ptr(), st if T > 1 else Hkv * d


def attn_kv4_append(k: torch.Tensor, v: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor,
                    seq_lens: torch.Tensor, cu_new: torch.Tensor, page_size: int, k_out: torch.Tensor | None = None,
                    v_out: torch.Tensor | None = None, stream=None) -> None:
    """Quantizes bf16 k and v [num_new, Hkv, d] (any token stride) into the 4-bit pool: rows
    cu_new[s]..cu_new[s+1]-1 are the last tokens of sequence s, whose length seq_lens[s] includes them.
    k_out and v_out (bf16 [num_new, Hkv, d]) receive the values the cache then stands for."""
    lib = _LIB or load_library()
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("k must be a torch.Tensor [num_new, Hkv, d]")
    dev = _current_device()
    shape = k.shape
    T, Hkv, d = shape
    kp, ks = _token_rows(k, "k", shape, dev)
    vp, vs = _token_rows(v, "v", shape, dev)
    (pool, table, lens), S, pool_heads, num_pages, max_pages = _kv4_pool(kv_pool, block_table, seq_lens, page_size, d,
                                                                         dev)
    if pool_heads != Hkv:
        raise ValueError("k and kv_pool must have the same number of KV heads")
    cu = _ptr(cu_new, "cu_new", torch.int32, 1, dev)
    if cu_new.shape[0] != S + 1:
        raise ValueError("cu_new must be [num_seqs + 1]")
    ko = None if k_out is None else _ptr(k_out, "k_out", torch.bfloat16, 3, dev)
    vo = None if v_out is None else _ptr(v_out, "v_out", torch.bfloat16, 3, dev)
    if (ko is not None and k_out.shape != shape) or (vo is not None and v_out.shape != shape):
        raise ValueError("k_out and v_out must be [num_new, Hkv, d]")
    st = lib.attn_kv4_append(kp, vp, ks, vs, pool, table, lens, cu, page_size, ko, vo, S, T, Hkv, d, num_pages,
                             max_pages, _stream(stream))
    if st:
        _check(st, "attn_kv4_append")


def attn_kv4_gather(kv_pool: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, page_size: int,
                    k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Reads the first min(seq_lens[s], N) cached tokens of every sequence into bf16 k and v
    [num_seqs, Hkv, N, d] (attn_fwd's layout); rows past a sequence's end keep what they hold."""
    lib = _LIB or load_library()
    dev = _current_device()
    kp, vp = _ptr(k, "k", torch.bfloat16, 4, dev), _ptr(v, "v", torch.bfloat16, 4, dev)
    rows, heads, N, d = k.shape
    (pool, table, lens), S, Hkv, num_pages, max_pages = _kv4_pool(kv_pool, block_table, seq_lens, page_size, d, dev)
    if rows != S or heads != Hkv or v.shape != k.shape:
        raise ValueError("k and v must be [num_seqs, Hkv, N, d]")
    st = lib.attn_kv4_gather(pool, table, lens, page_size, kp, vp, S, Hkv, N, d, num_pages, max_pages,
                             _stream(stream))
    if st:
        _check(st, "attn_kv4_gather")


def attn_decode_paged_kv4_workspace_size(num_seqs: int, Hq: int, Hkv: int, d: int) -> int:
    return int(load_library().attn_decode_paged_kv4_workspace_size(num_seqs, Hq, Hkv, d))


def attn_decode_paged_kv4(q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                          page_size: int, o: torch.Tensor, lse: torch.Tensor | None, scale: float,
                          workspace: torch.Tensor, stream=None) -> None:
    """One decode step over a 4-bit paged cache: q and o bf16 [num_seqs, Hq, d], lse fp32 [num_seqs, Hq] or None."""
    lib = _LIB or load_library()
    dev = _current_device()
    qp, op = _ptr(q, "q", torch.bfloat16, 3, dev), _ptr(o, "o", torch.bfloat16, 3, dev)
    shape = q.shape
    S, Hq, d = shape
    (pool, table, lens), rows, Hkv, num_pages, max_pages = _kv4_pool(kv_pool, block_table, seq_lens, page_size, d, dev)
    if rows != S:
        raise ValueError("block_table must be [num_seqs, max_pages_per_seq] with q's num_seqs")
    if o.shape != shape:
        raise ValueError("o must be [num_seqs, Hq, d]")
    lp = None
    if lse is not None:
        lp = _ptr(lse, "lse", torch.float32, 2, dev)
        if lse.shape != (S, Hq):
            raise ValueError("lse must be [num_seqs, Hq]")
    ws, nbytes = _scratch(workspace, dev)
    st = lib.attn_decode_paged_kv4(qp, pool, table, lens, page_size, op, lp, S, Hq, Hkv, d, num_pages, max_pages,
                                   scale, ws, nbytes, _stream(stream))
    if st:
        _check(st, "attn_decode_paged_kv4")


def _page_pools(pools, dev: int) -> tuple:
    """Checks pools that share a table: (pointer array, count, bytes per page, num_pages)."""
    if len(pools) == 0:
        raise ValueError("pools must hold at least one tensor [num_pages, ...]")
    first = pools[0]
    if not isinstance(first, torch.Tensor) or first.dim() < 2:
        raise TypeError("a pool must be a torch.Tensor [num_pages, ...]")
    num_pages, nbytes = first.shape[0], first.nbytes
    ptrs = (ctypes.c_void_p * len(pools))()
    for i, p in enumerate(pools):
        ptrs[i] = _ptr(p, "a pool", p.dtype, p.dim(), dev)
        if p.dim() < 2 or p.shape[0] != num_pages or p.nbytes != nbytes:
            raise ValueError("pools must be [num_pages, ...] with the same number and size of pages")
    return ptrs, len(pools), nbytes // num_pages if num_pages else 0, num_pages


def attn_pages_workspace_size(num_pages: int, rows: int) -> int:
    return int(load_library().attn_pages_workspace_size(num_pages, rows))


def attn_pages_fork(block_table: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor,
                    add_tokens: torch.Tensor | None, new_table: torch.Tensor, new_lens: torch.Tensor, page_size: int,
                    pools: list[torch.Tensor], workspace: torch.Tensor, n_free: torch.Tensor | None = None,
                    stream=None) -> None:
    """Builds new_table and new_lens: row i continues row parents[i] of the old table (-1: empty) with
    add_tokens[i] tokens more (or fewer).  Full pages are shared, a part-filled last page is copied for
    all but one of the rows that continue it (in every pool), new pages come from the free ones."""
    lib = _LIB or load_library()
    dev, i32 = _current_device(), torch.int32
    args = (_ptr(block_table, "block_table", i32, 2, dev), _ptr(seq_lens, "seq_lens", i32, 1, dev),
            _ptr(parents, "parents", i32, 1, dev),
            None if add_tokens is None else _ptr(add_tokens, "add_tokens", i32, 1, dev),
            _ptr(new_table, "new_table", i32, 2, dev), _ptr(new_lens, "new_lens", i32, 1, dev))
    S, cols = block_table.shape
    rows, new_cols = new_table.shape
    if seq_lens.shape[0] != S or parents.shape[0] != rows or new_lens.shape[0] != rows or \
            (add_tokens is not None and add_tokens.shape[0] != rows):
        raise ValueError("seq_lens must be [num_seqs]; parents, add_tokens and new_lens [new_rows]")
    if n_free is not None and n_free.numel() != 1:
        raise ValueError("n_free must hold one number")
    ptrs, n, page_bytes, num_pages = _page_pools(pools, dev)
    ws, nbytes = _scratch(workspace, dev)
    st = lib.attn_pages_fork(*args, page_size, ptrs, n, page_bytes, S, cols, rows, new_cols, num_pages,
                             None if n_free is None else _ptr(n_free, "n_free", i32, n_free.dim(), dev), ws, nbytes,
                             _stream(stream))
    if st:
        _check(st, "attn_pages_fork")


def attn_pages_compact(block_table: torch.Tensor, seq_lens: torch.Tensor, new_table: torch.Tensor,
                       page_map: torch.Tensor, page_size: int, pools: list[torch.Tensor], workspace: torch.Tensor,
                       n_live: torch.Tensor | None = None, stream=None) -> None:
    """Renumbers the n pages in use to 0..n-1, moving their contents in every pool: new_table (may be
    block_table) and page_map int32 [num_pages] (new number of each page, -1: free)."""
    lib = _LIB or load_library()
    dev, i32 = _current_device(), torch.int32
    args = (_ptr(block_table, "block_table", i32, 2, dev), _ptr(seq_lens, "seq_lens", i32, 1, dev),
            _ptr(new_table, "new_table", i32, 2, dev), _ptr(page_map, "page_map", i32, 1, dev))
    S, cols = block_table.shape
    if seq_lens.shape[0] != S or new_table.shape != block_table.shape:
        raise ValueError("seq_lens must be [num_seqs] and new_table [num_seqs, max_pages_per_seq]")
    if n_live is not None and n_live.numel() != 1:
        raise ValueError("n_live must hold one number")
    ptrs, n, page_bytes, num_pages = _page_pools(pools, dev)
    if page_map.shape[0] != num_pages:
        raise ValueError("page_map must be [num_pages]")
    ws, nbytes = _scratch(workspace, dev)
    st = lib.attn_pages_compact(*args, page_size, ptrs, n, page_bytes, S, cols, num_pages,
                                None if n_live is None else _ptr(n_live, "n_live", i32, n_live.dim(), dev), ws, nbytes,
                                _stream(stream))
    if st:
        _check(st, "attn_pages_compact")


def attn_get_device_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the first fault a kernel latched."""
    return int(load_library().attn_get_device_status(_stream(stream)))


def attn_debug_watchdog(timeout_ns: int, stream=None) -> None:
    _check(load_library().attn_debug_watchdog(int(timeout_ns), _stream(stream)), "attn_debug_watchdog")


def attn_debug_fwd_stall(q, k, v, o, lse, causal: bool, scale: float, stall_cta: int, stall_fill: int,
                         timeout_ns: int, stream=None) -> None:
    """attn_fwd_ex with one K/V ring fill left out in one CTA and pipeline waits limited to
    timeout_ns: exercises the kernel's timeout wind-down (testing only)."""
    lib = load_library()
    ptrs, dims = _fwd_shapes(q, k, v, o, lse)
    st = lib.attn_debug_fwd_stall(*ptrs, *dims, float(scale), int(bool(causal)), int(stall_cta), int(stall_fill),
                                  int(timeout_ns), _stream(stream))
    _check(st, "attn_debug_fwd_stall")


def attn_debug_bwd_stall(q, k, v, o, do, lse, dq, dk, dv, causal: bool, scale: float, stall_cta: int,
                         stall_step: int, timeout_ns: int, workspace: torch.Tensor | None = None, stream=None) -> None:
    """attn_bwd with the Q tile of one step left out in one CTA of the gradient kernel and
    pipeline waits limited to timeout_ns (testing only)."""
    args = _bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, scale, workspace)
    st = load_library().attn_debug_bwd_stall(*args, int(stall_cta), int(stall_step), int(timeout_ns), _stream(stream))
    _check(st, "attn_debug_bwd_stall")


def attn_debug_decode_stall(q, k_pool, v_pool, block_table, seq_lens, page_size: int, o, lse, scale: float,
                            workspace: torch.Tensor, stall_cta: int, stall_piece: int, timeout_ns: int,
                            stream=None) -> None:
    """attn_decode_paged with one K/V piece left out in one CTA of the split kernel and
    pipeline waits limited to timeout_ns (testing only)."""
    lib = load_library()
    S, Hq, d = q.shape
    num_pages, Hkv, ps, d2 = k_pool.shape
    if ps != page_size or d2 != d or tuple(v_pool.shape) != tuple(k_pool.shape):
        raise ValueError("pools must be [num_pages, Hkv, page_size, d]")
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError("block_table must be [num_seqs, max_pages_per_seq]")
    st = lib.attn_debug_decode_stall(
        _dev(q, "q", torch.bfloat16, 3), _dev(k_pool, "k_pool", torch.bfloat16, 4),
        _dev(v_pool, "v_pool", torch.bfloat16, 4), _dev(block_table, "block_table", torch.int32, 2),
        _dev(seq_lens, "seq_lens", torch.int32, 1), page_size, _dev(o, "o", torch.bfloat16, 3),
        None if lse is None else _dev(lse, "lse", torch.float32, 2), S, Hq, Hkv, d, num_pages,
        block_table.shape[1], float(scale), _dev(workspace, "workspace", workspace.dtype),
        workspace.numel() * workspace.element_size(), int(stall_cta), int(stall_piece), int(timeout_ns),
        _stream(stream))
    _check(st, "attn_debug_decode_stall")


def attn_debug_exp2(x: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """y = 2^x by the kernel's FMA-pipe polynomial (fp32 device tensors)."""
    n = x.numel()
    if y.numel() != n:
        raise ValueError("x and y must have the same size")
    _check(load_library().attn_debug_exp2(_dev(x, "x", torch.float32), _dev(y, "y", torch.float32), n,
                                          _stream(stream)), "attn_debug_exp2")


def attn_status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()
