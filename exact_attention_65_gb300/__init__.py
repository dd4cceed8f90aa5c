"""exact_attention_65_gb300: exact attention on one GB300 through the exattn C ABI.

A thin ctypes binding over ``libexattn.so`` (built by
``exact_attention_65_gb300.build``). It only checks and marshals arguments:
every step of the computation runs in the library's CUDA kernels, and there
is no CPU or framework fallback. PyTorch supplies device memory and the
current CUDA stream.

    o, lse = attn_fwd(q, k, v)                  # q, k, v: [b, s, h, d] fp16/bf16 CUDA tensors
    o, lse = attn_decode_splitkv(q, k, v)       # split-KV decode, num_splits=0: heuristic
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libexattn.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "exattn.h")

ATTN_FP16, ATTN_BF16 = 0, 1
ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_NO_MEMORY = 4
ATTN_ERR_DEVICE_TIMEOUT = 5
ATTN_DEBUG_SKIP_LOADS = 1
ATTN_DEBUG_GENERAL_FWD = 2
ATTN_DEBUG_GENERAL_BWD = 4

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    """A non-OK status returned by the C ABI."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {attn_status_string(status)} (status {status})")


def load_library() -> ctypes.CDLL:
    """Load libexattn.so; raise if it has not been built (there is no fallback)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m exact_attention_65_gb300.build` (there is no CPU fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, f32, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint
        lib.attn_fwd.restype = i32
        lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp]
        lib.attn_decode_splitkv.restype = i32
        lib.attn_decode_splitkv.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp]
        lib.attn_decode_splitkv_ex.restype = i32
        lib.attn_decode_splitkv_ex.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32,
                                               i32, i32, vp]
        lib.attn_fwd_host.restype = i32
        lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, i32, vp]
        lib.attn_fwd_causal.restype = i32
        lib.attn_fwd_causal.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp]
        lib.attn_decode_splitkv_causal.restype = i32
        lib.attn_decode_splitkv_causal.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                                   f32, i32, i32, vp]
        lib.attn_decode_paged.restype = i32
        lib.attn_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                          i32, f32, i32, i32, vp]
        lib.attn_decode_paged_ex.restype = i32
        lib.attn_decode_paged_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                             i32, i32, f32, i32, i32, i32, vp]
        for fn in (lib.attn_bwd, lib.attn_bwd_causal):
            fn.restype = i32
            fn.argtypes = [vp] * 9 + [i32, i32, i32, i32, i32, f32, i32, vp]
        i64 = ctypes.c_int64
        lib.attn_fwd_packed.restype = i32
        lib.attn_fwd_packed.argtypes = [vp] * 7 + [i32] * 7 + [i64] * 3 + [f32, i32, i32, vp]
        lib.attn_bwd_packed.restype = i32
        lib.attn_bwd_packed.argtypes = [vp] * 11 + [i32] * 6 + [i64] * 6 + [f32, i32, i32, vp]
        lib.attn_chunk_paged.restype = i32
        lib.attn_chunk_paged.argtypes = [vp] * 8 + [i32] * 9 + [i64, f32, i32, i32, vp]
        lib.attn_paged_plan.restype = i32
        lib.attn_paged_plan.argtypes = [vp] * 9 + [i32] * 4 + [i64, vp]
        lib.attn_paged_write.restype = i32
        lib.attn_paged_write.argtypes = [vp] * 5 + [i64] + [i32] * 4 + [i64] * 2 + [i32, vp]
        lib.attn_paged_append.restype = i32
        lib.attn_paged_append.argtypes = [vp] * 9 + [i64] * 2 + [i32] * 7 + [i64] * 4 + [i32, vp]
        lib.attn_paged_append_q4.restype = i32
        lib.attn_paged_append_q4.argtypes = [vp] * 9 + [i64] * 2 + [i32] * 7 + [i64] * 4 + [f32] * 2 + [i32, vp]
        lib.attn_paged_read_q4.restype = i32
        lib.attn_paged_read_q4.argtypes = [vp] * 5 + [i64] + [i32] * 4 + [f32] * 2 + [i64] * 2 + [i32, vp]
        lib.attn_chunk_paged_q4.restype = i32
        lib.attn_chunk_paged_q4.argtypes = [vp] * 8 + [i32] * 9 + [i64] + [f32] * 3 + [i32, i32, vp]
        lib.attn_q4_page_bytes.restype = i64
        lib.attn_q4_page_bytes.argtypes = [i32] * 2
        lib.attn_debug_packed_plan.restype = i32
        lib.attn_debug_packed_plan.argtypes = [vp, vp] + [i32] * 8 + [vp]
        lib.attn_debug_few_plan.restype = i32
        lib.attn_debug_few_plan.argtypes = [vp, vp] + [i32] * 7 + [vp]
        lib.attn_debug_packed_starts.restype = i32
        lib.attn_debug_packed_starts.argtypes = [vp, vp] + [i32] * 10 + [vp]
        lib.attn_debug_packed_shares.restype = i32
        lib.attn_debug_packed_shares.argtypes = [vp, vp] + [i32] * 5 + [vp]
        lib.attn_decode_splitkv_noalloc.restype = i32
        lib.attn_decode_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                                    f32, i32, i32, vp]
        lib.attn_get_noalloc_status.restype = i32
        lib.attn_get_noalloc_status.argtypes = [vp]
        lib.attn_decode_num_splits.restype = i32
        lib.attn_decode_num_splits.argtypes = [i32] * 5
        lib.attn_decode_num_splits_for_sms.restype = i32
        lib.attn_decode_num_splits_for_sms.argtypes = [i32] * 6
        lib.attn_get_device_status.restype = i32
        lib.attn_get_device_status.argtypes = [vp]
        lib.attn_last_timeout_site.restype = u32
        lib.attn_last_timeout_site.argtypes = []
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_status_string.argtypes = [i32]
        lib.attn_release_workspace.restype = None
        lib.attn_release_workspace.argtypes = []
        lib.attn_debug_set_flags.restype = None
        lib.attn_debug_set_flags.argtypes = [u32]
        lib.attn_version.restype = i32
        lib.attn_version.argtypes = []
        _lib = lib
        return lib


def attn_status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()


_DTYPE_CODE = {torch.float16: ATTN_FP16, torch.bfloat16: ATTN_BF16}
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _dtype_code(t: torch.Tensor) -> int:
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"exattn takes float16 or bfloat16 tensors, got {t.dtype}")
    return code


def _check_slow(q, k, v):
    """Raises the specific error for a q, k, v triple _check refused."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [b, s, h, d], got shape {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous in (b, s, h, d) order")
    raise ValueError("invalid q, k, v")


def _check(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    """Sizes (b, sq, sk, h, d), dtype code and device index of a q, k, v
    triple; raises on anything the C ABI would not take. Kept lean: small
    problems issue in a few microseconds, and this runs on every call."""
    try:
        ok = (q.is_cuda and k.is_cuda and v.is_cuda and q.dim() == 4 and k.dim() == 4
              and v.dim() == 4 and q.is_contiguous() and k.is_contiguous() and v.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        _check_slow(q, k, v)
    dt = q.dtype
    if k.dtype is not dt or v.dtype is not dt:
        raise TypeError("q, k, v must share one dtype")
    idx = q.get_device()
    if k.get_device() != idx or v.get_device() != idx:
        raise ValueError("q, k, v must be on the same device")
    b, sq, h, d = q.shape
    kb, sk, kh, kd = k.shape
    if kb != b or kh != h or kd != d or v.shape != k.shape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    code = _DTYPE_CODE.get(dt)
    if code is None:
        raise TypeError(f"exattn takes float16 or bfloat16 tensors, got {dt}")
    return b, sq, sk, h, d, code, idx


def _empty(shape, dtype, device, stream):
    """A result made by the call, in memory of the stream that writes it: what
    the current stream gave back may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):  # (anything with a cuda_stream will do for a call)
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _outputs(q, out, lse, b, h, sq, idx, stream):
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    elif (out.shape != q.shape or out.dtype is not q.dtype or not out.is_contiguous()
          or out.get_device() != idx):
        raise ValueError("out must be a contiguous tensor like q")
    if lse is None:
        lse = _empty((b, h, sq), torch.float32, q.device, stream)
    elif (lse.shape != (b, h, sq) or lse.dtype is not torch.float32 or not lse.is_contiguous()
          or lse.get_device() != idx):
        raise ValueError("lse must be a contiguous float32 tensor [b, h, sq]")
    return out, lse


def _stream(device, stream):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _call(fn, idx, stream, *args):
    """Call C-ABI function ``fn`` with ``args`` plus the stream, with device
    ``idx`` current. The common case (device already current, its current
    stream) skips the device context manager and the Stream object."""
    if idx == _current_device():
        raw = _current_raw_stream(idx) if stream is None else stream.cuda_stream
        return fn(*args, raw)
    device = torch.device("cuda", idx)
    with torch.cuda.device(device):
        return fn(*args, _stream(device, stream))


def attn_fwd(q, k, v, scale: float | None = None, out=None, lse=None, stream=None,
             causal: bool = False):
    """Exact attention O = softmax(scale * Q K^T) V and LSE [b, h, sq] (fp32).

    q: [b, sq, h, d], k/v: [b, sk, h, d], fp16 or bf16, contiguous CUDA
    tensors; default scale 1/sqrt(d). Runs on ``stream`` (default: the
    current stream of q's device); results that are not given are made on
    that stream, as if it were current. ``causal``: bottom-right-aligned mask
    (query row i sees key j only if j <= i + sk - sq)."""
    b, sq, sk, h, d, dt, idx = _check(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    out, lse = _outputs(q, out, lse, b, h, sq, idx, stream)
    lib = _lib or load_library()
    fn = lib.attn_fwd_causal if causal else lib.attn_fwd
    rc = _call(fn, idx, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
               lse.data_ptr(), b, sq, sk, h, d, scale, dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_causal" if causal else "attn_fwd")
    return out, lse


def attn_fwd_host(q, k, v, scale: float | None = None, out=None, lse=None, causal: bool = False,
                  device=None, stream=None, sync: bool = True):
    """attn_fwd on host (CPU) tensors through the library's copy / compute /
    copy-back pipeline (attn_fwd_host in the C ABI).

    q: [b, sq, h, d], k/v: [b, sk, h, d], fp16 or bf16, contiguous CPU
    tensors, best in pinned memory (pageable ones work, without overlap).
    out and lse (CPU) are allocated pinned when not given. Runs on
    ``device`` (default: the current CUDA device) and ``stream`` (its
    current stream). With ``sync`` False the call returns once the work is
    queued: out and lse are valid, and the inputs may be reused, only after
    the stream is synchronised."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
            raise ValueError(f"{name} must be a CPU tensor (attn_fwd takes CUDA tensors)")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [b, s, h, d] tensor")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    b, sq, h, d = q.shape
    if k.shape != v.shape or k.shape[0] != b or k.shape[2] != h or k.shape[3] != d:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    dt = _dtype_code(q)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.device.type != "cpu":
        raise ValueError("out must be a contiguous CPU tensor like q")
    if lse is None:
        lse = torch.empty((b, h, sq), dtype=torch.float32, pin_memory=True)
    elif (tuple(lse.shape) != (b, h, sq) or lse.dtype != torch.float32 or not lse.is_contiguous()
          or lse.device.type != "cpu"):
        raise ValueError("lse must be a contiguous float32 CPU tensor [b, h, sq]")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    lib = load_library()
    with torch.cuda.device(device):
        st = _stream(device, stream)
        rc = lib.attn_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               lse.data_ptr(), b, sq, k.shape[1], h, d, scale, dt, 1 if causal else 0, st)
        if rc != ATTN_OK:
            raise AttnError(rc, "attn_fwd_host")
        if sync:
            (torch.cuda.current_stream(device) if stream is None else stream).synchronize()
    return out, lse


def attn_decode_splitkv(q, k, v, scale: float | None = None, num_splits: int = 0, out=None,
                        lse=None, stream=None, causal: bool = False):
    """Split-KV decode: same result as attn_fwd, computed by splitting the
    keys into ``num_splits`` ranges (0 = heuristic) and reducing the
    per-split (O_i, LSE_i) with the log-sum-exp combine."""
    b, sq, sk, h, d, dt, idx = _check(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    out, lse = _outputs(q, out, lse, b, h, sq, idx, stream)
    lib = _lib or load_library()
    fn = lib.attn_decode_splitkv_causal if causal else lib.attn_decode_splitkv_ex
    rc = _call(fn, idx, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
               lse.data_ptr(), b, sq, sk, h, d, scale, int(num_splits), dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_splitkv")
    return out, lse


def attn_decode_paged(q, k_pages, v_pages, block_table, seqlens_k, scale: float | None = None,
                      num_splits: int = 0, out=None, lse=None, stream=None, causal: bool = False):
    """Split-KV decode of the new rows of each sequence from a paged KV cache.

    q: [b, sq, h, d] (sq new rows per sequence); k_pages, v_pages:
    [num_pages, page_size, h, d] (page_size a multiple of 16); block_table:
    int32 [b, max_pages] pool page of each logical page; seqlens_k: int32
    [b] keys per sequence. All CUDA tensors. ``causal``: the
    bottom-right-aligned mask against each sequence's own key count."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 4:
        raise ValueError("q must be a CUDA tensor [b, sq, h, d]")
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor [num_pages, page_size, h, d]")
        if t.dtype != q.dtype or t.device != q.device:
            raise ValueError(f"{name} must match q's dtype and device")
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    for name, t in (("block_table", block_table), ("seqlens_k", seqlens_k)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda \
                or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor on q's device")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    b, sq, h, d = q.shape
    num_pages, page_size = k_pages.shape[0], k_pages.shape[1]
    if k_pages.shape[2] != h or k_pages.shape[3] != d:
        raise ValueError("page pools must be [num_pages, page_size, h, d] with q's h and d")
    if block_table.dim() != 2 or block_table.shape[0] != b or tuple(seqlens_k.shape) != (b,):
        raise ValueError("block_table must be [b, max_pages] and seqlens_k [b]")
    dt = _dtype_code(q)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    idx = q.get_device()
    out, lse = _outputs(q, out, lse, b, h, sq, idx, stream)
    lib = _lib or load_library()
    rc = _call(lib.attn_decode_paged_ex, idx, stream, q.data_ptr(), k_pages.data_ptr(),
               v_pages.data_ptr(), block_table.data_ptr(), seqlens_k.data_ptr(), out.data_ptr(),
               lse.data_ptr(), b, sq, h, d, num_pages, page_size, block_table.shape[1], scale,
               int(num_splits), 1 if causal else 0, dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_paged")
    return out, lse


def attn_bwd(q, k, v, o, lse, dout, scale: float | None = None, dq=None, dk=None, dv=None,
             stream=None, causal: bool = False):
    """Backward pass of attn_fwd: returns (dq, dk, dv).

    q, o, dout: [b, sq, h, d]; k, v: [b, sk, h, d] (fp16 or bf16, contiguous
    CUDA tensors); lse: fp32 [b, h, sq] from attn_fwd with the same
    ``causal`` (the bottom-right-aligned mask, attn_bwd_causal)."""
    b, sq, sk, h, d, dt, idx = _check(q, k, v)
    for name, t in (("o", o), ("dout", dout)):
        if not isinstance(t, torch.Tensor) or t.shape != q.shape or t.dtype != q.dtype \
                or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous tensor like q")
    if (tuple(lse.shape) != (b, h, sq) or lse.dtype != torch.float32 or not lse.is_contiguous()
            or lse.device != q.device):
        raise ValueError("lse must be a contiguous float32 tensor [b, h, sq]")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = (_empty(x.shape, x.dtype, x.device, stream) if t is None else t
                  for t, x in ((dq, q), (dk, k), (dv, v)))
    for name, t, ref in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t.shape != ref.shape or t.dtype != ref.dtype or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous tensor like {name[1]}")
    lib = _lib or load_library()
    fn = lib.attn_bwd_causal if causal else lib.attn_bwd
    rc = _call(fn, idx, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
               lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
               b, sq, sk, h, d, scale, dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_causal" if causal else "attn_bwd")
    return dq, dk, dv


_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _rows(name, t, idx, dt):
    """Token stride of packed rows [tokens, heads, d] whose heads lie side by
    side (a tensor of their own, or a slice of wider rows)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a CUDA tensor [tokens, heads, d] (there is no CPU path)")
    if t.dtype is not dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}: all rows share one dtype")
    if t.get_device() != idx:
        raise ValueError(f"{name} must be on the same device as the other tensors")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if s2 == 1 and (s1 == d or h == 1) and s0 >= h * d and s0 % 8 == 0:
        return s0
    # (a lone row has no distance to the next one)
    if not t.is_contiguous():
        raise ValueError(f"{name}: heads must lie d apart within a token's row, and rows a multiple of 8 apart")
    return h * d


def _array(name, t, shape, idx, dtype):
    """Raises if t is not a contiguous array of that shape and dtype on device idx."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != idx \
            or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor {list(shape)} on the same device")


def _packed_q(q, cu_seqlens_q, out, lse, stream):
    """Sizes, dtype code, device index and token stride of packed query rows,
    with their outputs. (Kept lean: short batches issue in a few microseconds,
    and this runs on every call.)"""
    try:
        idx = q.get_device()
        dt = q.dtype
        t, h, d = q.shape
        s0, s1, s2 = q.stride()
        b = cu_seqlens_q.shape[0] - 1
        fine = (idx >= 0 and s2 == 1 and s1 == d and s0 >= h * d and s0 % 8 == 0 and cu_seqlens_q.dtype is _I32
                and cu_seqlens_q.get_device() == idx and cu_seqlens_q.is_contiguous()
                and cu_seqlens_q.dim() == 1 and b >= 1)
    except (AttributeError, ValueError, TypeError, IndexError):
        fine = False
    if not fine:
        if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
            raise ValueError("q must be a CUDA tensor [total_q, h, d] (there is no CPU path)")
        idx, dt = q.get_device(), q.dtype
        t, h, d = q.shape
        s0 = _rows("q", q, idx, dt)
        if not isinstance(cu_seqlens_q, torch.Tensor) or cu_seqlens_q.dim() != 1 or cu_seqlens_q.shape[0] < 2:
            raise ValueError("cu_seqlens_q must be an int32 tensor [b + 1]")
        b = cu_seqlens_q.shape[0] - 1
        _array("cu_seqlens_q", cu_seqlens_q, (b + 1,), idx, _I32)
    code = _DTYPE_CODE.get(dt)
    if code is None:
        raise TypeError(f"exattn takes float16 or bfloat16 tensors, got {dt}")
    if out is None:
        out = _empty((t, h, d), dt, q.device, stream)
    elif out.shape != q.shape or out.dtype is not dt or not out.is_contiguous() or out.get_device() != idx:
        raise ValueError("out must be a contiguous tensor with q's shape and dtype")
    if lse is None:
        lse = _empty((h, t), _F32, q.device, stream)
    elif (lse.shape != (h, t) or lse.dtype is not _F32 or not lse.is_contiguous()
          or lse.get_device() != idx):
        raise ValueError("lse must be a contiguous float32 tensor [h, total_q]")
    return b, t, h, d, code, idx, s0, out, lse


def _packed_kv(q, k, v, cu_seqlens_k, b, h, d, idx):
    """Rows, heads and token strides of packed k and v."""
    try:
        dt = q.dtype
        tk, hk, dk = k.shape
        ks, k1, k2 = k.stride()
        vs, v1, v2 = v.stride()
        row = hk * d
        fine = (k.dtype is dt and v.dtype is dt and k.get_device() == idx and v.get_device() == idx
                and v.shape == k.shape and dk == d and k2 == 1 and v2 == 1 and k1 == d and v1 == d and ks >= row
                and vs >= row and ks % 8 == 0 and vs % 8 == 0 and hk >= 1 and h % hk == 0
                and cu_seqlens_k.dtype is _I32 and cu_seqlens_k.get_device() == idx
                and cu_seqlens_k.shape == (b + 1,) and cu_seqlens_k.is_contiguous())
    except (AttributeError, ValueError, TypeError):
        fine = False
    if not fine:
        ks, vs = _rows("k", k, idx, q.dtype), _rows("v", v, idx, q.dtype)
        tk, hk, dk = k.shape
        if v.shape != k.shape or dk != d or hk < 1 or h % hk:
            raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
        _array("cu_seqlens_k", cu_seqlens_k, (b + 1,), idx, _I32)
    return tk, hk, ks, vs


def attn_fwd_packed(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int = 0,
                    scale: float | None = None, out=None, lse=None, stream=None, causal: bool = False):
    """Attention over sequences of different lengths packed one behind the
    other, with grouped heads.

    q: [total_q, h, d], k/v: [total_k, h_kv, d], fp16 or bf16 CUDA tensors, h
    a multiple of h_kv; each may be a slice of wider rows (any token stride,
    heads side by side). cu_seqlens_q, cu_seqlens_k: int32 [b + 1], sequence i
    holds rows cu[i] .. cu[i + 1] - 1. max_seqlen_q: the most rows a sequence
    has (0: not known, taken as total_q). It only picks the kernel's form, but
    give it for short sequences: where none has more than 128 h_kv / h rows a
    call without it can take half as long again. ``causal``: the
    bottom-right-aligned mask of each sequence's own lengths. Returns out
    [total_q, h, d] and lse [h, total_q]; rows of no sequence are left as
    they were. Outputs may not overlap inputs or each other."""
    b, t, h, d, dt, idx, qs, out, lse = _packed_q(q, cu_seqlens_q, out, lse, stream)
    tk, hk, ks, vs = _packed_kv(q, k, v, cu_seqlens_k, b, h, d, idx)
    lib = _lib or load_library()
    rc = _call(lib.attn_fwd_packed, idx, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(),
               cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), out.data_ptr(), lse.data_ptr(), b, t, tk,
               max_seqlen_q, h, hk, d, qs, ks, vs, 1.0 / math.sqrt(d) if scale is None else float(scale),
               1 if causal else 0, dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_packed")
    return out, lse


def attn_bwd_packed(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, scale: float | None = None,
                    dq=None, dk=None, dv=None, stream=None, causal: bool = False):
    """Backward pass of attn_fwd_packed: returns (dq, dk, dv).

    q, k, v, cu_seqlens_q, cu_seqlens_k, ``causal``: as in the forward; o,
    lse: its results; dout: [total_q, h, d], contiguous. dq, dk, dv may be
    slices of wider rows, as q, k, v may (tensors of their own where they are
    not given); rows of no sequence are left as they were."""
    if o is None or lse is None:
        raise ValueError("o and lse must be the forward's results")
    b, t, h, d, dt, idx, qs, o, lse = _packed_q(q, cu_seqlens_q, o, lse, stream)
    tk, hk, ks, vs = _packed_kv(q, k, v, cu_seqlens_k, b, h, d, idx)
    if not isinstance(dout, torch.Tensor) or dout.shape != q.shape or dout.dtype is not q.dtype \
            or not dout.is_contiguous() or dout.get_device() != idx:
        raise ValueError("dout must be a contiguous tensor with q's shape and dtype")
    grads, strides = [], []
    for name, x, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if x is None:
            x = _empty(like.shape, like.dtype, like.device, stream)
        strides.append(_rows(name, x, idx, q.dtype))
        if x.shape != like.shape:
            raise ValueError(f"{name} must have {name[1]}'s shape")
        grads.append(x)
    lib = _lib or load_library()
    rc = _call(lib.attn_bwd_packed, idx, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
               lse.data_ptr(), dout.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
               grads[0].data_ptr(), grads[1].data_ptr(), grads[2].data_ptr(), b, t, tk, h, hk, d, qs, ks, vs,
               *strides, 1.0 / math.sqrt(d) if scale is None else float(scale), 1 if causal else 0, dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_packed")
    return tuple(grads)


def _pools(k_pages, v_pages, idx, dt):
    """Shape [num_pages, page_size, h_kv, d] of a pair of page pools."""
    try:
        shape = k_pages.shape
        fine = (len(shape) == 4 and v_pages.shape == shape and k_pages.dtype is dt and v_pages.dtype is dt
                and k_pages.get_device() == idx and v_pages.get_device() == idx and k_pages.is_contiguous()
                and v_pages.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not isinstance(t, torch.Tensor) or t.dim() != 4 or t.get_device() != idx or t.dtype is not dt \
                    or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous tensor [num_pages, page_size, h_kv, d] with the "
                                 "rows' dtype and device")
        raise ValueError("k_pages and v_pages must have the same shape")
    return shape


def attn_chunk_paged(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q: int = 0,
                     scale: float | None = None, out=None, lse=None, stream=None, causal: bool = False):
    """Attention of each request's new tokens (one, or a chunk of a prompt)
    over a paged KV cache that holds them already, with grouped heads.

    q: [total_q, h, d], request i's rows cu_seqlens_q[i] .. cu_seqlens_q[i +
    1] - 1 (int32 [b + 1]); k_pages, v_pages: [num_pages, page_size, h_kv, d]
    (page_size a multiple of 16); block_table: int32 [b, max_pages];
    seqlens_k: int32 [b] keys per request with the new ones. ``causal``: the
    bottom-right-aligned mask against each request's own key count. Other
    arguments and results as attn_fwd_packed (max_seqlen_q: 64 requests with a
    token each take 150 us with it and 221 without)."""
    b, t, h, d, dt, idx, qs, out, lse = _packed_q(q, cu_seqlens_q, out, lse, stream)
    num_pages, page_size, hk, dk = _pools(k_pages, v_pages, idx, q.dtype)
    if dk != d or hk < 1 or h % hk:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, pages {tuple(k_pages.shape)}")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be an int32 tensor [b, max_pages]")
    max_pages = block_table.shape[1]
    _array("block_table", block_table, (b, max_pages), idx, _I32)
    _array("seqlens_k", seqlens_k, (b,), idx, _I32)
    lib = _lib or load_library()
    rc = _call(lib.attn_chunk_paged, idx, stream, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
               block_table.data_ptr(), cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), out.data_ptr(),
               lse.data_ptr(), b, t, max_seqlen_q, h, hk, d, num_pages, page_size, max_pages, qs,
               1.0 / math.sqrt(d) if scale is None else float(scale), 1 if causal else 0, dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_chunk_paged")
    return out, lse


def attn_paged_plan(seqlens_k, new_lens, block_table, free_pages, free_count, page_size: int,
                    max_tokens: int | None = None, cu_seqlens_q=None, seqlens_out=None, slot_map=None,
                    free_left=None, stream=None):
    """Block tables and slot maps of one step, built on the device.

    seqlens_k: int32 [b] keys in the cache; new_lens: int32 [b] tokens each
    request brings; block_table: int32 [b, max_pages], updated in place with
    the pages taken; free_pages: int32 [num_free], a stack whose first
    free_count (int32 [1]) entries are free. slot_map has max_tokens entries
    (needed unless slot_map is given): a bound on the step's new tokens that
    the host knows. Returns (cu_seqlens_q [b + 1], seqlens_out [b], slot_map
    int64 [max_tokens], free_left [1]); a negative free_left says how many
    pages were lacking. Inputs are left as they are: seqlens_out and
    free_left are the next step's seqlens_k and free_count.

    The caller sees to two things: a request with more keys than its table
    row holds (seqlens_out below seqlens_k + new_lens) or more new tokens than
    max_tokens leave tokens without a slot, and such a step must not be run.
    A finished request's pages go back by writing its table's entries behind
    the first free_count of free_pages and raising the count."""
    if not isinstance(seqlens_k, torch.Tensor) or not seqlens_k.is_cuda or seqlens_k.dim() != 1:
        raise ValueError("seqlens_k must be an int32 CUDA tensor [b] (there is no CPU path)")
    b, idx = seqlens_k.shape[0], seqlens_k.get_device()
    if cu_seqlens_q is None:
        cu_seqlens_q = _empty(b + 1, _I32, seqlens_k.device, stream)
    if seqlens_out is None:
        seqlens_out = _empty(b, _I32, seqlens_k.device, stream)
    if free_left is None:
        free_left = _empty(1, _I32, seqlens_k.device, stream)
    if slot_map is None:
        if max_tokens is None:
            raise ValueError("give max_tokens or slot_map")
        slot_map = _empty(int(max_tokens), _I64, seqlens_k.device, stream)
    elif max_tokens is not None and int(max_tokens) != slot_map.numel():
        raise ValueError("slot_map must have max_tokens entries")
    for name, t, n in (("block_table", block_table, 2), ("free_pages", free_pages, 1), ("slot_map", slot_map, 1)):
        if not isinstance(t, torch.Tensor) or t.dim() != n:
            raise ValueError(f"{name} must be a tensor of {n} dimension(s)")
    max_pages, num_free, room = block_table.shape[1], free_pages.shape[0], slot_map.shape[0]
    for name, t, shape in (("seqlens_k", seqlens_k, (b,)), ("new_lens", new_lens, (b,)),
                           ("block_table", block_table, (b, max_pages)), ("free_pages", free_pages, (num_free,)),
                           ("free_count", free_count, (1,)), ("cu_seqlens_q", cu_seqlens_q, (b + 1,)),
                           ("seqlens_out", seqlens_out, (b,)), ("free_left", free_left, (1,))):
        try:
            fine = t.dtype is _I32 and t.get_device() == idx and t.shape == shape and t.is_contiguous()
        except AttributeError:
            fine = False
        if not fine:
            _array(name, t, shape, idx, _I32)
    _array("slot_map", slot_map, (room,), idx, _I64)
    lib = _lib or load_library()
    rc = _call(lib.attn_paged_plan, idx, stream, seqlens_k.data_ptr(), new_lens.data_ptr(),
               block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), cu_seqlens_q.data_ptr(),
               seqlens_out.data_ptr(), slot_map.data_ptr(), free_left.data_ptr(), b, max_pages, page_size,
               num_free, room)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_paged_plan")
    return cu_seqlens_q, seqlens_out, slot_map, free_left


def attn_paged_write(k, v, slot_map, k_pages, v_pages, stream=None):
    """New K and V rows into the pages of a paged cache.

    k, v: [tokens, h_kv, d] (each may be a slice of wider rows); slot_map:
    int64 [tokens], the row of token t in the pools seen as [num_pages *
    page_size, h_kv, d] (attn_paged_plan's; slots outside the pools, such as
    -1, are skipped); k_pages, v_pages: [num_pages, page_size, h_kv, d],
    written in place. Rows that move within the pools may not lie in slots
    that the call writes."""
    if not isinstance(k, torch.Tensor) or not k.is_cuda or k.dim() != 3:
        raise ValueError("k must be a CUDA tensor [tokens, h_kv, d] (there is no CPU path)")
    idx, dt = k.get_device(), k.dtype
    code = _dtype_code(k)
    ks, vs = _rows("k", k, idx, dt), _rows("v", v, idx, dt)
    num_pages, page_size, hk, d = _pools(k_pages, v_pages, idx, dt)
    t, h, dk = k.shape
    if v.shape != k.shape or h != hk or dk != d:
        raise ValueError(f"shape mismatch: k {tuple(k.shape)}, v {tuple(v.shape)}, pages {tuple(k_pages.shape)}")
    _array("slot_map", slot_map, (t,), idx, _I64)
    lib = _lib or load_library()
    rc = _call(lib.attn_paged_write, idx, stream, k.data_ptr(), v.data_ptr(), slot_map.data_ptr(),
               k_pages.data_ptr(), v_pages.data_ptr(), t, hk, d, num_pages, page_size, ks, vs, code)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_paged_write")


def _append_args(q, k, v, cos_sin, positions, slot_map, q_out, stream):
    """Sizes, strides, dtype code and device index of an append's rows, with
    its output. (Kept lean: a decode step's append issues in a few microseconds.)"""
    try:
        idx, dt = q.get_device(), q.dtype
        t, h, d = q.shape
        tk, hk, dk = k.shape
        qs, q1, q2 = q.stride()
        ks, k1, k2 = k.stride()
        vs, v1, v2 = v.stride()
        if q_out is None:
            q_out = _empty((t, h, d), dt, q.device, stream)
        os, o1, o2 = q_out.stride()
        far, rot = cos_sin.shape
        row, krow = h * d, hk * d
        fine = (idx >= 0 and k.dtype is dt and v.dtype is dt and q_out.dtype is dt and cos_sin.dtype is _F32
                and positions.dtype is _I64 and slot_map.dtype is _I64 and k.get_device() == idx
                and v.get_device() == idx and q_out.get_device() == idx and cos_sin.get_device() == idx
                and positions.get_device() == idx and slot_map.get_device() == idx and v.shape == k.shape
                and tk == t and dk == d and q_out.shape == q.shape and positions.shape == (t,)
                and slot_map.shape == (t,) and q2 == 1 and k2 == 1 and v2 == 1 and o2 == 1 and q1 == d and k1 == d
                and v1 == d and o1 == d and qs >= row and os >= row and ks >= krow and vs >= krow
                and (qs | os | ks | vs) % 8 == 0 and cos_sin.is_contiguous() and positions.is_contiguous()
                and slot_map.is_contiguous())
    except (AttributeError, ValueError, TypeError):
        fine = False
    if not fine:
        if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
            raise ValueError("q must be a CUDA tensor [tokens, h, d] (there is no CPU path)")
        idx, dt = q.get_device(), q.dtype
        qs, ks, vs = _rows("q", q, idx, dt), _rows("k", k, idx, dt), _rows("v", v, idx, dt)
        t, h, d = q.shape
        hk = k.shape[1]
        if k.shape != v.shape or k.shape[0] != t or k.shape[2] != d:
            raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
        if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
            raise ValueError("cos_sin must be a float32 tensor [max_positions, rot]")
        far, rot = cos_sin.shape
        _array("cos_sin", cos_sin, (far, rot), idx, _F32)
        _array("positions", positions, (t,), idx, _I64)
        _array("slot_map", slot_map, (t,), idx, _I64)
        if q_out is None:
            q_out = _empty((t, h, d), dt, q.device, stream)
        os = _rows("q_out", q_out, idx, dt)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    code = _DTYPE_CODE.get(dt)
    if code is None:
        raise TypeError(f"exattn takes float16 or bfloat16 tensors, got {dt}")
    return t, h, hk, d, far, rot, qs, ks, vs, os, code, idx, q_out


def attn_paged_append(q, k, v, cos_sin, positions, slot_map, k_pages, v_pages, q_out=None,
                      interleaved: bool = False, stream=None):
    """A step's queries and keys rotated by their positions, keys and values
    into the pages of a paged cache; returns the rotated queries.

    q: [tokens, h, d], k, v: [tokens, h_kv, d] (each may be a slice of wider
    rows); cos_sin: float32 [max_positions, rot], row p the cosines of the rot /
    2 angles of position p and then their sines; the first rot channels of a
    head turn (a multiple of 16); positions: int64 [tokens]; slot_map: int64
    [tokens] as in attn_paged_write (a token with a slot outside the pools is
    not stored, but its queries are rotated; for a position that cos_sin does
    not have nothing is written). ``interleaved``: channels 2 i and 2 i + 1 are
    a pair, instead of i and i + rot / 2. q_out: [tokens, h, d], also a slice
    of wider rows, or q itself. k_pages, v_pages: [num_pages, page_size, h_kv,
    d], written in place; they may not overlap the rows."""
    t, h, hk, d, far, rot, qs, ks, vs, os, code, idx, q_out = _append_args(q, k, v, cos_sin, positions, slot_map,
                                                                         q_out, stream)
    num_pages, page_size, ph, pd = _pools(k_pages, v_pages, idx, q.dtype)
    if ph != hk or pd != d:
        raise ValueError(f"shape mismatch: k {tuple(k.shape)}, pages {tuple(k_pages.shape)}")
    lib = _lib or load_library()
    rc = _call(lib.attn_paged_append, idx, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), cos_sin.data_ptr(),
               positions.data_ptr(), slot_map.data_ptr(), q_out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
               t, far, rot, 1 if interleaved else 0, h, hk, d, num_pages, page_size, qs,
               ks, vs, os, code)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_paged_append")
    return q_out


def attn_q4_page_bytes(page_size: int, d: int) -> int:
    """Bytes of a page of one head of a 4-bit cache (0: not supported)."""
    return load_library().attn_q4_page_bytes(page_size, d)


def _pools_q4(k_pages, v_pages, d, idx):
    """(num_pages, h_kv, page_size) of a pair of 4-bit pools of head dim d."""
    try:
        shape = k_pages.shape
        num_pages, h, block = shape
        fine = (k_pages.dtype is torch.uint8 and v_pages.dtype is torch.uint8 and v_pages.shape == shape
                and k_pages.get_device() == idx and v_pages.get_device() == idx and k_pages.is_contiguous()
                and v_pages.is_contiguous())
    except (AttributeError, ValueError, TypeError):
        fine = False
    if not fine:
        raise ValueError("k_pages and v_pages must be contiguous uint8 tensors [num_pages, h_kv, page_size * 9 d / 16] "
                         "of one shape on the rows' device")
    # 9 d / 16 bytes of a row and head
    if d < 16 or block % (9 * d // 16):
        raise ValueError(f"pages {tuple(shape)} do not hold whole rows of head dim {d}")
    return num_pages, h, block // (9 * d // 16)


def attn_paged_append_q4(q, k, v, cos_sin, positions, slot_map, k_pages, v_pages, k_scale: float = 1.0,
                         v_scale: float = 1.0, q_out=None, interleaved: bool = False, stream=None):
    """attn_paged_append into a cache held in 4 bits; returns the rotated queries.

    k_pages, v_pages: uint8 [num_pages, h_kv, page_size * 9 d / 16]
    (attn_q4_page_bytes(page_size, d)), page_size a multiple of 16: per page
    and head, rows of e2m1 codes (two to a byte) and then rows of e4m3 scales,
    one for 16 channels. A value is code * scale * k_scale (v_scale); every
    call on a pool gets the same scales."""
    t, h, hk, d, far, rot, qs, ks, vs, os, code, idx, q_out = _append_args(q, k, v, cos_sin, positions, slot_map,
                                                                         q_out, stream)
    num_pages, ph, page_size = _pools_q4(k_pages, v_pages, d, idx)
    if ph != hk:
        raise ValueError(f"shape mismatch: k {tuple(k.shape)}, pages {tuple(k_pages.shape)}")
    lib = _lib or load_library()
    rc = _call(lib.attn_paged_append_q4, idx, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), cos_sin.data_ptr(),
               positions.data_ptr(), slot_map.data_ptr(), q_out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
               t, far, rot, 1 if interleaved else 0, h, hk, d, num_pages, page_size, qs,
               ks, vs, os, k_scale, v_scale, code)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_paged_append_q4")
    return q_out


def attn_chunk_paged_q4(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q: int = 0,
                        scale: float | None = None, k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None,
                        stream=None, causal: bool = False):
    """attn_chunk_paged over a cache held in 4 bits: attention of each
    request's new tokens over the values that its pages hold, with grouped heads.

    k_pages, v_pages, k_scale, v_scale: as in attn_paged_append_q4, which put
    the new tokens' own rows there. max_seqlen_q: the most tokens a request
    brings, 0 if not known; give it (64 requests with four tokens each over up
    to 8192 keys, h32 on 8, take 95 us with it and 199 without). Other arguments
    and results as attn_chunk_paged."""
    b, t, h, d, dt, idx, qs, out, lse = _packed_q(q, cu_seqlens_q, out, lse, stream)
    num_pages, hk, page_size = _pools_q4(k_pages, v_pages, d, idx)
    if hk < 1 or h % hk:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, pages {tuple(k_pages.shape)}")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be an int32 tensor [b, max_pages]")
    max_pages = block_table.shape[1]
    _array("block_table", block_table, (b, max_pages), idx, _I32)
    _array("seqlens_k", seqlens_k, (b,), idx, _I32)
    lib = _lib or load_library()
    rc = _call(lib.attn_chunk_paged_q4, idx, stream, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
               block_table.data_ptr(), cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), out.data_ptr(),
               lse.data_ptr(), b, t, max_seqlen_q, h, hk, d, num_pages, page_size, max_pages, qs,
               1.0 / math.sqrt(d) if scale is None else float(scale), k_scale, v_scale, 1 if causal else 0, dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_chunk_paged_q4")
    return out, lse


def attn_paged_read_q4(k_pages, v_pages, slot_map, d: int, dtype=torch.bfloat16, k_scale: float = 1.0,
                       v_scale: float = 1.0, k=None, v=None, stream=None):
    """Rows of a 4-bit cache in 16 bits: returns k, v [tokens, h_kv, d].

    k_pages, v_pages, k_scale, v_scale: as in attn_paged_append_q4; slot_map:
    int64 [tokens], the slot of each row (zeros come back for one outside the
    pools). k, v may be given (then dtype is theirs), also as slices of wider
    rows."""
    if not isinstance(slot_map, torch.Tensor) or not slot_map.is_cuda or slot_map.dim() != 1:
        raise ValueError("slot_map must be an int64 CUDA tensor [tokens] (there is no CPU path)")
    idx, t = slot_map.get_device(), slot_map.shape[0]
    _array("slot_map", slot_map, (t,), idx, _I64)
    num_pages, h, page_size = _pools_q4(k_pages, v_pages, d, idx)
    given = k if k is not None else v
    if given is not None:
        if not isinstance(given, torch.Tensor):
            raise ValueError("k and v must be CUDA tensors [tokens, h_kv, d]")
        dtype = given.dtype
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise TypeError(f"exattn takes float16 or bfloat16 tensors, got {dtype}")
    if k is None:
        k = _empty((t, h, d), dtype, slot_map.device, stream)
    if v is None:
        v = _empty((t, h, d), dtype, slot_map.device, stream)
    ks, vs = _rows("k", k, idx, dtype), _rows("v", v, idx, dtype)
    if tuple(k.shape) != (t, h, d) or v.shape != k.shape:
        raise ValueError(f"k and v must be [{t}, {h}, {d}]")
    lib = _lib or load_library()
    rc = _call(lib.attn_paged_read_q4, idx, stream, k_pages.data_ptr(), v_pages.data_ptr(), slot_map.data_ptr(),
               k.data_ptr(), v.data_ptr(), t, h, d, num_pages, page_size, k_scale, v_scale, ks, vs, code)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_paged_read_q4")
    return k, v


def attn_decode_splitkv_noalloc(q, k, v, out, lse, scale: float | None = None,
                                num_splits: int = 0, stream=None):
    """attn_decode_splitkv for callers that cannot allocate device memory:
    out and lse must be given, and the per-split partials live in a fixed
    array inside the library (calls that overlap on the GPU race on it).
    Its kernels' timeouts are read by attn_get_noalloc_status()."""
    b, sq, sk, h, d, dt, idx = _check(q, k, v)
    if out is None or lse is None:
        raise ValueError("out and lse must be given: this entry point allocates nothing")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    out, lse = _outputs(q, out, lse, b, h, sq, idx, stream)
    lib = _lib or load_library()
    rc = _call(lib.attn_decode_splitkv_noalloc, idx, stream, q.data_ptr(), k.data_ptr(),
               v.data_ptr(), out.data_ptr(), lse.data_ptr(), b, sq, sk, h, d, scale,
               int(num_splits), dt)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_splitkv_noalloc")
    return out, lse


def attn_get_noalloc_status(stream=None, device=None) -> int:
    """Synchronise the stream and return (and clear) the status word of the
    no-allocation decode."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(device):
        return load_library().attn_get_noalloc_status(_stream(device, stream))


def attn_decode_num_splits(b: int, sq: int, sk: int, h: int, d: int) -> int:
    """Split count the heuristic picks on the current device."""
    return load_library().attn_decode_num_splits(b, sq, sk, h, d)


def attn_decode_num_splits_for_sms(b: int, sq: int, sk: int, h: int, d: int, num_sms: int) -> int:
    """Split count the heuristic picks for a device with ``num_sms`` SMs."""
    return load_library().attn_decode_num_splits_for_sms(b, sq, sk, h, d, num_sms)


def attn_get_device_status(stream=None, device=None) -> int:
    """Synchronise the stream and return (and clear) the device status."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(device):
        return load_library().attn_get_device_status(_stream(device, stream))


def attn_last_timeout_site() -> int:
    return load_library().attn_last_timeout_site()


def attn_release_workspace() -> None:
    load_library().attn_release_workspace()


def attn_debug_set_flags(flags: int) -> None:
    load_library().attn_debug_set_flags(int(flags))


__all__ = [
    "AttnError", "attn_fwd", "attn_fwd_host", "attn_bwd", "attn_decode_splitkv",
    "attn_decode_paged", "attn_fwd_packed", "attn_bwd_packed", "attn_chunk_paged", "attn_paged_plan", "attn_paged_write",
    "attn_paged_append", "attn_paged_append_q4", "attn_paged_read_q4", "attn_chunk_paged_q4",
    "attn_q4_page_bytes",
    "attn_decode_splitkv_noalloc", "attn_get_noalloc_status",
    "attn_decode_num_splits",
    "attn_decode_num_splits_for_sms", "attn_get_device_status", "attn_last_timeout_site",
    "attn_release_workspace", "attn_debug_set_flags", "attn_status_string", "load_library",
]
