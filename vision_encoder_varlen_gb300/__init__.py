"""GB300 (sm_103a) varlen ViT encoder attention: thin Python binding of libvitattn.

Argument marshalling only: every step runs in the library's CUDA kernels,
reached through its C ABI (include/vit_attn.h). PyTorch provides device
memory and the current stream. There is no CPU or eager fallback: if the
library is not built, every call raises.

    inv_freq, pos_hw, cu = rope_freqs(grid_hw, T, head_dim)       # 2D RoPE table + positions
    qk_norm_rope(q, k, pos_hw, inv_freq, norm_w, eps, inplace=True)
    out = varlen_attn(q, k, v, cu, max_seqlen)                    # [T, H, D] bf16
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libvitattn.so")
MAX_SEGMENTS = 8192
HEAD_DIMS = (32, 64, 80, 96, 128)

_lock = threading.Lock()
_lib = None


def _declare_block(L):
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    rope = [vp, vp, vp, i32, i32, vp, f32]      # pos, inv_freq, sections, axis layout, rope mode, norm_w, eps
    for name, args in (
            ("vit_grid_positions", [vp, i32, i64, vp, vp, vp, vp]),
            ("vit_qk_norm_mrope", [vp] * 4 + [i64, i32, i32, i32] + [i64] * 4 + rope + [vp]),
            ("vit_qk_norm_mrope_bwd", [vp] * 6 + [i64, i32, i32, i32] + [i64] * 6 + rope + [vp, vp, sz, vp]),
            ("vit_cross_attn", [vp] * 3 + [i64, i64, i32, i32, i32] + [i64] * 3 + [vp] * 3 + [i32, i32, i32, f32, vp,
                                                                                              i64, vp, vp, sz, vp, vp]),
            ("vit_cross_attn_bwd", [vp] * 6 + [i64, i64, i32, i32, i32] + [i64] * 5 + [vp] * 3 + [i32, i32, i32, f32] +
             [vp] * 3 + [i64] * 3 + [i32, vp, sz, vp, vp]),
            ("vit_window_attn", [vp] * 3 + [i64, i64, i32, i32, i32] + [i64] * 3 + [vp] * 3 + [i32] * 5 +
             [f32, vp, i64, vp, vp, sz, vp, vp]),
            ("vit_window_attn_bwd", [vp] * 6 + [i64, i64, i32, i32, i32] + [i64] * 5 + [vp] * 3 + [i32] * 5 + [f32] +
             [vp] * 3 + [i64] * 3 + [i32, vp, sz, vp, vp]),
            ("vit_prefix_attn", [vp] * 5 + [i64] * 3 + [i32] * 3 + [i64] * 5 + [vp] * 5 + [i32] * 5 +
             [f32, vp, i64, vp, vp, sz, vp, vp]),
            ("vit_norm_residual", [vp] * 7 + [i64, i32, i32] + [i64] * 5 + [f32, f32, vp]),
            ("vit_norm_residual_bwd", [vp] * 12 + [i64, i32, i32] + [i64] * 8 + [f32, f32, vp, sz, vp, vp])):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, i32
    for name, args in (("vit_qk_norm_mrope_bwd_workspace_size", [i32]),
                       ("vit_cross_attn_workspace_size", [i64, i64] + [i32] * 6),
                       ("vit_cross_attn_bwd_workspace_size", [i64, i64] + [i32] * 6),
                       ("vit_window_attn_workspace_size", [i64, i64] + [i32] * 8),
                       ("vit_window_attn_bwd_workspace_size", [i64, i64] + [i32] * 8),
                       ("vit_prefix_attn_workspace_size", [i64] * 3 + [i32] * 8),
                       ("vit_norm_residual_bwd_workspace_size", [i32])):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, sz


class VitError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} (status {code})")


class _QRope(ctypes.Structure):
    _fields_ = [("pos_hw", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int),
                ("norm_w", ctypes.c_void_p), ("eps", ctypes.c_float), ("rope_mode", ctypes.c_int)]


class _AttnOptions(ctypes.Structure):
    _fields_ = [("short_segment_max", ctypes.c_int)]


class _KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


def lib() -> ctypes.CDLL:
    """The loaded libvitattn (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                                   "g.build()'` (needs nvcc); there is no fallback implementation")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
            L.vit_version.restype = ctypes.c_char_p
            L.vit_status_string.restype = ctypes.c_char_p
            L.vit_status_string.argtypes = [i32]
            L.vit_device_supported.argtypes = [i32]
            L.vit_rope_freqs.argtypes = [i32, f32, vp, i32, i64, vp, vp, vp, vp, vp]
            L.vit_qk_norm_rope.argtypes = [vp, vp, vp, vp, i64, i32, i32, i64, i64, i64, i64, vp, vp, vp, f32, vp]
            L.vit_qk_norm_rope_ex.argtypes = [vp, vp, vp, vp, i64, i32, i32, i64, i64, i64, i64, vp, vp, vp, f32,
                                              i32, vp, vp]
            L.vit_varlen_attn_workspace_size.restype = sz
            L.vit_varlen_attn_workspace_size.argtypes = [i64, i32, i32, i32]
            L.vit_varlen_attn.argtypes = [vp, vp, vp, i64, i32, i32, i64, i64, i64, vp, i32, i32, f32, vp, i64, vp,
                                          sz, vp, vp]
            L.vit_varlen_attn_lse.argtypes = [vp, vp, vp, i64, i32, i32, i64, i64, i64, vp, i32, i32, f32, vp, i64,
                                              vp, vp, sz, vp, vp]
            L.vit_varlen_attn_fused_q.argtypes = [vp, vp, vp, i64, i32, i32, i64, i64, i64, ctypes.POINTER(_QRope),
                                                  vp, i32, i32, f32, vp, i64, vp, vp, sz, vp, vp]
            L.vit_rope_table.argtypes = [vp, i32, i32, vp, vp]
            L.vit_varlen_attn_padded.argtypes = [vp, vp, vp, i64, i32, i32, i64, i64, i64, vp, vp, i32, i32, f32, vp,
                                                 i64, vp, ctypes.POINTER(_QRope), vp, sz, vp, vp]
            L.vit_varlen_attn_ex.argtypes = [vp, vp, vp, i64, i32, i32, i64, i64, i64, vp, vp, vp, i32, i32, f32, vp,
                                             i64, vp, ctypes.POINTER(_QRope), ctypes.POINTER(_AttnOptions), vp, sz,
                                             vp, vp]
            L.vit_read_status.argtypes = [vp, vp]
            L.vit_launch_count.restype = i64
            L.vit_kernel_timing.argtypes = [i32]
            L.vit_kernel_timing_read.argtypes = [ctypes.POINTER(_KernelTime), i32]
            _declare_block(L)
            for fn in ("vit_device_supported", "vit_rope_freqs", "vit_qk_norm_rope", "vit_qk_norm_rope_ex",
                       "vit_varlen_attn", "vit_varlen_attn_lse", "vit_varlen_attn_fused_q", "vit_rope_table",
                       "vit_varlen_attn_padded", "vit_varlen_attn_ex",
                       "vit_read_status", "vit_kernel_timing", "vit_kernel_timing_read"):
                getattr(L, fn).restype = i32
            _lib = L
    return _lib


_tls = threading.local()


@contextlib.contextmanager
def kernel_split(short_max: int | None):
    """Within the block, attention calls made by this thread pass ``short_max`` as their kernel
    split (segments longer than min(short_max, 64) run on the tcgen05 kernel, the others on the
    tiny-segment kernel); None restores the library default.
    Per thread, and passed with every call: the library itself keeps no setting between calls."""
    prev = getattr(_tls, "short_max", None)
    _tls.short_max = None if short_max is None else int(short_max)
    try:
        yield
    finally:
        _tls.short_max = prev


def _split(short_max):
    return short_max if short_max is not None else getattr(_tls, "short_max", None)


def status_string(code: int) -> str:
    return lib().vit_status_string(int(code)).decode()


def version() -> str:
    return lib().vit_version().decode()


def _check(code: int, what: str):
    if code != 0:
        raise VitError(code, what)


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _tok_stride(t: torch.Tensor, name: str, H: int, D: int) -> int:
    if t.dim() != 3 or t.shape[1] != H or t.shape[2] != D:
        raise ValueError(f"{name} must be [T, {H}, {D}], got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
    if t.stride(2) != 1 or t.stride(1) != D:
        raise ValueError(f"{name} needs head stride D and unit element stride (got strides {t.stride()})")
    return t.stride(0)


def new_status(device=None) -> torch.Tensor:
    """A zeroed device status word for the device-detected errors of the calls."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def read_status(status: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return the status word (0 = ok)."""
    code = lib().vit_read_status(_ptr(status), _stream(stream))
    return int(code)


def rope_freqs(grid_hw: torch.Tensor, total_tokens: int, head_dim: int, theta: float = 10000.0, *,
               status: torch.Tensor | None = None, stream=None):
    """2D RoPE frequency table (dim = head_dim/2), per-token (row, col) and cu_seqlens from a device grid list."""
    if grid_hw.dtype != torch.int32 or not grid_hw.is_cuda or not grid_hw.is_contiguous():
        raise ValueError("grid_hw must be a contiguous CUDA int32 tensor [n_img, 2]")
    n = grid_hw.numel() // 2
    dev = grid_hw.device
    dim = head_dim // 2
    inv_freq = torch.empty(dim // 2, dtype=torch.float32, device=dev)
    pos = torch.empty((total_tokens, 2), dtype=torch.int32, device=dev)
    cu = torch.empty(n + 1, dtype=torch.int32, device=dev)
    _check(lib().vit_rope_freqs(dim, float(theta), _ptr(grid_hw), n, int(total_tokens), _ptr(inv_freq), _ptr(pos),
                                _ptr(cu), _ptr(status), _stream(stream)), "vit_rope_freqs")
    return inv_freq, pos, cu


def rope_table(inv_freq: torch.Tensor, head_dim: int, max_pos: int, *, stream=None) -> torch.Tensor:
    """cos/sin of p * inv_freq for positions p < max_pos (fp32 [max_pos, head_dim/2]), the table the
    fused-Q attention rotates with."""
    if inv_freq.dtype != torch.float32 or not inv_freq.is_cuda or inv_freq.numel() != head_dim // 4:
        raise ValueError(f"inv_freq must be a CUDA float32 tensor [{head_dim // 4}]")
    cs = torch.empty((int(max_pos), head_dim // 2), dtype=torch.float32, device=inv_freq.device)
    _check(lib().vit_rope_table(_ptr(inv_freq), int(head_dim), int(max_pos), _ptr(cs), _stream(stream)),
           "vit_rope_table")
    return cs


ROPE_ROTATE_HALF = 0    # pairs (m, m + D/2)
ROPE_INTERLEAVED = 1    # pairs (2m, 2m + 1), the "complex_rope" mode


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, pos_hw: torch.Tensor, inv_freq: torch.Tensor,
                 norm_w: torch.Tensor | None = None, eps: float = 1e-6, *, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None, inplace: bool = False, interleaved: bool = False,
                 status: torch.Tensor | None = None, stream=None):
    """QK-RMSNorm (if norm_w [2, D] is given) + 2D RoPE. Returns (q', k'); a half passed as None is
    skipped and returned as None. ``interleaved`` rotates adjacent pairs instead of (m, m + D/2)."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("at least one of q and k is required")
    T, H, D = ref.shape
    qs = _tok_stride(q, "q", H, D) if q is not None else 0
    ks = _tok_stride(k, "k", H, D) if k is not None else 0
    if q is not None and k is not None and q.shape[0] != k.shape[0]:
        raise ValueError("q and k must have the same number of tokens")
    if inplace:
        q_out, k_out = q, k
    if q is not None and q_out is None:
        q_out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    if k is not None and k_out is None:
        k_out = torch.empty((T, H, D), dtype=k.dtype, device=k.device)
    if q is None:
        q_out = None
    if k is None:
        k_out = None
    qos = _tok_stride(q_out, "q_out", H, D) if q_out is not None else 0
    kos = _tok_stride(k_out, "k_out", H, D) if k_out is not None else 0
    if norm_w is not None and (norm_w.dtype != torch.bfloat16 or norm_w.numel() != 2 * D
                               or not norm_w.is_contiguous()):
        raise ValueError("norm_w must be a contiguous bfloat16 tensor [2, D]")
    mode = ROPE_INTERLEAVED if interleaved else ROPE_ROTATE_HALF
    _check(lib().vit_qk_norm_rope_ex(_ptr(q), _ptr(q_out), _ptr(k), _ptr(k_out), T, H, D, qs, qos, ks, kos,
                                     _ptr(pos_hw), _ptr(inv_freq), _ptr(norm_w), float(eps), mode, _ptr(status),
                                     _stream(stream)),
           "vit_qk_norm_rope_ex")
    return q_out, k_out


def workspace_size(T: int, H: int, B: int, D: int) -> int:
    return int(lib().vit_varlen_attn_workspace_size(int(T), *_ints(H, B, D)))


def _c_int(x: int) -> int:
    """x as a C int: the nearest one where x passes 32 bits, of which ctypes would keep the low ones without a word."""
    return max(-2 ** 31, min(x, 2 ** 31 - 1))


def _ints(*x) -> tuple:
    return tuple(_c_int(int(v)) for v in x)


def _max_seqlen(m) -> int:
    """The C convention: 0 = not given (the library bounds the segments by T)."""
    return 0 if m is None else _c_int(int(m))


def _attn_ex(q, k, v, qs, ks, vs, cu_seqlens, seq_start, seq_len, B, max_seqlen, scale, out, os_, lse, qr,
             short_max, workspace, status, stream, what):
    opts = _AttnOptions(_c_int(int(short_max)))
    _check(lib().vit_varlen_attn_ex(_ptr(q), _ptr(k), _ptr(v), q.shape[0], q.shape[1], q.shape[2], qs, ks, vs,
                                    _ptr(cu_seqlens), _ptr(seq_start), _ptr(seq_len), B, _max_seqlen(max_seqlen),
                                    float(scale) if scale is not None else 0.0, _ptr(out), os_, _ptr(lse),
                                    ctypes.byref(qr) if qr is not None else None, ctypes.byref(opts),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
                                    _stream(stream)), what)


def varlen_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor | None,
                max_seqlen: int | None = None, scale: float | None = None, *, num_segments: int | None = None,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                status: torch.Tensor | None = None, return_lse: bool = False, lse: torch.Tensor | None = None,
                short_max: int | None = None, stream=None):
    """Non-causal attention inside each packed segment. q, k, v [T, H, D] bf16 -> out [T, H, D] bf16.

    ``max_seqlen`` bounds the segment lengths (a padded bucket is fine); None leaves the bound
    to the library (T), so nothing is read back to the host. With ``return_lse`` (or an ``lse``
    buffer) also returns lse [T, H] fp32, the natural-log sum of exp(scale * q.k) over each
    row's segment: (out, lse). ``short_max`` is this call's kernel split (see kernel_split)."""
    T, H, D = q.shape
    qs, ks, vs = _tok_stride(q, "q", H, D), _tok_stride(k, "k", H, D), _tok_stride(v, "v", H, D)
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous CUDA int32 tensor [B + 1]")
        B = cu_seqlens.numel() - 1
    else:
        if num_segments is None:
            raise ValueError("num_segments is required when cu_seqlens is None")
        B = _c_int(int(num_segments))
    if out is None:
        out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    os_ = _tok_stride(out, "out", H, D)
    need = workspace_size(T, H, B, D)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    sc = float(scale) if scale is not None else 0.0
    ws_bytes = workspace.numel() * workspace.element_size()
    short_max = _split(short_max)
    if return_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (T, H) or not lse.is_contiguous()
                            or not lse.is_cuda):
        raise ValueError(f"lse must be a contiguous CUDA float32 tensor [{T}, {H}]")
    if short_max is not None:
        _attn_ex(q, k, v, qs, ks, vs, cu_seqlens, None, None, B, max_seqlen, scale, out, os_, lse, None, short_max,
                 workspace, status, stream, "vit_varlen_attn_ex")
        return (out, lse) if lse is not None else out
    if lse is None:
        _check(lib().vit_varlen_attn(_ptr(q), _ptr(k), _ptr(v), T, H, D, qs, ks, vs, _ptr(cu_seqlens), B,
                                     _max_seqlen(max_seqlen), sc, _ptr(out), os_, _ptr(workspace), ws_bytes,
                                     _ptr(status), _stream(stream)), "vit_varlen_attn")
        return out
    _check(lib().vit_varlen_attn_lse(_ptr(q), _ptr(k), _ptr(v), T, H, D, qs, ks, vs, _ptr(cu_seqlens), B,
                                     _max_seqlen(max_seqlen), sc, _ptr(out), os_, _ptr(lse), _ptr(workspace), ws_bytes,
                                     _ptr(status), _stream(stream)), "vit_varlen_attn_lse")
    return out, lse


def varlen_attn_fused_q(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor | None,
                        max_seqlen: int | None, pos_hw: torch.Tensor, cos_sin: torch.Tensor,
                        q_norm_w: torch.Tensor | None = None, eps: float = 1e-6, scale: float | None = None, *,
                        interleaved: bool = False, num_segments: int | None = None,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        status: torch.Tensor | None = None, return_lse: bool = False,
                        lse: torch.Tensor | None = None, short_max: int | None = None, stream=None):
    """varlen_attn on raw q: the kernels normalise (q_norm_w [D], or None) and rotate every Q tile
    after loading it. k must already be normalised and rotated (qk_norm_rope(None, k, ...))."""
    T, H, D = q.shape
    qs, ks, vs = _tok_stride(q, "q", H, D), _tok_stride(k, "k", H, D), _tok_stride(v, "v", H, D)
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous CUDA int32 tensor [B + 1]")
        B = cu_seqlens.numel() - 1
    else:
        if num_segments is None:
            raise ValueError("num_segments is required when cu_seqlens is None")
        B = _c_int(int(num_segments))
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or cos_sin.shape[1] != D // 2 \
            or not cos_sin.is_contiguous():
        raise ValueError(f"cos_sin must be the contiguous float32 [max_pos, {D // 2}] table of rope_table")
    if q_norm_w is not None and (q_norm_w.dtype != torch.bfloat16 or q_norm_w.numel() != D
                                 or not q_norm_w.is_contiguous()):
        raise ValueError("q_norm_w must be a contiguous bfloat16 tensor [D]")
    if out is None:
        out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    os_ = _tok_stride(out, "out", H, D)
    if workspace is None:
        workspace = torch.empty(max(workspace_size(T, H, B, D), 16), dtype=torch.uint8, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (T, H) or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous CUDA float32 tensor [{T}, {H}]")
    qr = _QRope(pos_hw.data_ptr(), cos_sin.data_ptr(), int(cos_sin.shape[0]),
                q_norm_w.data_ptr() if q_norm_w is not None else None, float(eps),
                ROPE_INTERLEAVED if interleaved else ROPE_ROTATE_HALF)
    short_max = _split(short_max)
    if short_max is not None:
        _attn_ex(q, k, v, qs, ks, vs, cu_seqlens, None, None, B, max_seqlen, scale, out, os_, lse, qr, short_max,
                 workspace, status, stream, "vit_varlen_attn_ex")
        return (out, lse) if lse is not None else out
    _check(lib().vit_varlen_attn_fused_q(_ptr(q), _ptr(k), _ptr(v), T, H, D, qs, ks, vs, ctypes.byref(qr),
                                         _ptr(cu_seqlens), B, _max_seqlen(max_seqlen),
                                         float(scale) if scale is not None else 0.0, _ptr(out), os_, _ptr(lse),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _ptr(status), _stream(stream)), "vit_varlen_attn_fused_q")
    return (out, lse) if lse is not None else out


def varlen_attn_padded(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seq_start: torch.Tensor,
                       seq_len: torch.Tensor, max_seqlen: int | None = None, scale: float | None = None, *,
                       out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       status: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       short_max: int | None = None, stream=None):
    """Attention over a padded layout: segment i is rows [seq_start[i], seq_start[i] + seq_len[i]) of
    q, k, v and out (ascending, not overlapping); rows between segments are left untouched. Nothing
    on the host depends on the lengths, so the call can be captured in a CUDA graph and replayed
    after new starts/lengths are written into the same device tensors."""
    T, H, D = q.shape
    qs, ks, vs = _tok_stride(q, "q", H, D), _tok_stride(k, "k", H, D), _tok_stride(v, "v", H, D)
    for name, t in (("seq_start", seq_start), ("seq_len", seq_len)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA int32 tensor [B]")
    B = seq_len.numel()
    if seq_start.numel() != B:
        raise ValueError("seq_start and seq_len must have the same length")
    if out is None:
        out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    os_ = _tok_stride(out, "out", H, D)
    if workspace is None:
        workspace = torch.empty(max(workspace_size(T, H, B, D), 16), dtype=torch.uint8, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (T, H) or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous CUDA float32 tensor [{T}, {H}]")
    short_max = _split(short_max)
    if short_max is not None:
        _attn_ex(q, k, v, qs, ks, vs, None, seq_start, seq_len, B, max_seqlen, scale, out, os_, lse, None, short_max,
                 workspace, status, stream, "vit_varlen_attn_ex")
        return out
    _check(lib().vit_varlen_attn_padded(_ptr(q), _ptr(k), _ptr(v), T, H, D, qs, ks, vs, _ptr(seq_start),
                                        _ptr(seq_len), B, _max_seqlen(max_seqlen),
                                        float(scale) if scale is not None else 0.0, _ptr(out), os_, _ptr(lse), None,
                                        _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)),
           "vit_varlen_attn_padded")
    return out


def encoder_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                 max_seqlen: int | None,
                 pos_hw: torch.Tensor, inv_freq: torch.Tensor, cos_sin: torch.Tensor,
                 norm_w: torch.Tensor | None = None, eps: float = 1e-6, *, interleaved: bool = False,
                 k_out: torch.Tensor | None = None, **kw):
    """The whole hot path with the Q prologue fused into attention: a one-tensor K pre-stage
    (norm_w row 1, written to k_out, or in place when k_out is k), then attention on raw q with
    norm_w row 0 applied as Q tiles load."""
    _, kr = qk_norm_rope(None, k, pos_hw, inv_freq, norm_w, eps, k_out=k_out, interleaved=interleaved,
                         stream=kw.get("stream"))
    q_w = norm_w.reshape(2, -1)[0] if norm_w is not None else None
    return varlen_attn_fused_q(q, kr, v, cu_seqlens, max_seqlen, pos_hw, cos_sin, q_w, eps,
                               interleaved=interleaved, **kw)


# ---- around a language model's reading of the encoder's states: three-axis rotary positions, cross
# ---- attention and the gated residual step with its norms, each with its gradient

def _device(*tensors) -> int:
    """The index of the one CUDA device that every tensor given is on."""
    dev = -1
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if dev < 0:
                dev = i
            if i < 0:
                raise ValueError("every tensor must be a CUDA tensor")
            if i != dev:
                raise ValueError(f"tensors on different devices: {dev} and {i}")
    return dev


def _call(fn: str, dev: int, stream, *args):
    """Calls a library function on device `dev`, on the caller's stream or the device's current one (the last
    argument of every function), and raises on an error."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    else:
        if stream.device_index != dev:
            raise ValueError(f"the stream is on device {stream.device_index}, the tensors on {dev}")
        handle = stream.cuda_stream
    f = getattr(lib(), fn)
    if torch.cuda.current_device() == dev:
        code = f(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = f(*args, handle)
    if code:
        raise VitError(code, fn)


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """A tensor on like's device that a call will write: from the pool of the stream the call is given (memory
    that the current stream has let go of may still be in use there), and marked as used on the current one."""
    dev = like.device
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)     # (half the time of like.new_empty)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _scratch(need: int, like: torch.Tensor, stream) -> torch.Tensor:
    return _new(like, max(need, 16), torch.uint8, stream)


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _rows3(t: torch.Tensor, name: str, T: int, H: int, D: int) -> int:
    """Token stride of bf16 [T, H, D] with head stride D."""
    if t.shape != (T, H, D):
        raise ValueError(f"{name} must be [{T}, {H}, {D}], got {tuple(t.shape)}")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
    st = t.stride()
    if st[2] != 1 or (st[1] != D and H > 1):
        raise ValueError(f"{name} needs head stride D and unit element stride (got strides {st})")
    return st[0] if T > 1 else H * D


def _shape3(t: torch.Tensor, name: str):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, D], got {tuple(t.shape)}")
    return t.shape


def grid_positions(grid_thw: torch.Tensor, total_tokens: int, *, status: torch.Tensor | None = None, stream=None):
    """Positions of packed images and clips: ([T, 3] int32 (frame, row, column), cu_seqlens [n + 1] int32) from
    a device list of (frames, rows, columns)."""
    if grid_thw.dtype is not _I32 or not grid_thw.is_contiguous() or grid_thw.dim() != 2 or grid_thw.shape[1] != 3:
        raise ValueError("grid_thw must be a contiguous CUDA int32 tensor [n, 3]")
    dev, n, T = _device(grid_thw, status), grid_thw.shape[0], int(total_tokens)
    if T < 0:
        raise ValueError("total_tokens must not be negative")
    pos, cu = _new(grid_thw, (T, 3), _I32, stream), _new(grid_thw, n + 1, _I32, stream)
    _call("vit_grid_positions", dev, stream, _addr(grid_thw), n, T, _addr(pos), _addr(cu), _word(status))
    return pos, cu


MROPE_BLOCKED = 0   # the sections one after the other
MROPE_CYCLED = 1    # time, height, width in turn


@functools.lru_cache(maxsize=64)
def _three(sections: tuple):
    return (ctypes.c_int * 3)(*map(_c_int, sections))


def _mrope_args(T, D, pos_thw, inv_freq, sections, norm_w, eps, cycled, interleaved):
    if pos_thw.dtype is not _I32 or pos_thw.shape != (T, 3) or not pos_thw.is_contiguous():
        raise ValueError(f"pos_thw must be a contiguous CUDA int32 tensor [{T}, 3]")
    if inv_freq.dtype is not _F32 or inv_freq.shape != (D // 2,) or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous CUDA float32 tensor [{D // 2}]")
    if norm_w is not None and (norm_w.dtype is not _BF16 or norm_w.shape != (2, D)
                               or not norm_w.is_contiguous()):
        raise ValueError(f"norm_w must be a contiguous CUDA bfloat16 tensor [2, {D}]")
    if len(sections) != 3:
        raise ValueError("sections must be three pair counts (time, height, width)")
    return (_addr(pos_thw), _addr(inv_freq), _three(tuple(sections)), MROPE_CYCLED if cycled else MROPE_BLOCKED,
            ROPE_INTERLEAVED if interleaved else ROPE_ROTATE_HALF, _addr(norm_w), float(eps))


def qk_norm_mrope(q: torch.Tensor | None, k: torch.Tensor | None, pos_thw: torch.Tensor, inv_freq: torch.Tensor,
                  sections, norm_w: torch.Tensor | None = None, eps: float = 1e-6, *, cycled: bool = False,
                  interleaved: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                  inplace: bool = False, stream=None):
    """QK-RMSNorm (if norm_w [2, D] is given) + rotary positions with three axes. q [T, Hq, D] and k [T, Hk, D]
    may differ in heads; a half passed as None is skipped and returned as None. ``sections`` are the pairs that
    follow time, height and width (their sum is D / 2), one after the other or, with ``cycled``, in turn."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("at least one of q and k is required")
    T, _, D = _shape3(ref, "q and k")
    if inplace:
        q_out, k_out = q, k
    dev = _device(q, k, q_out, k_out, pos_thw, inv_freq, norm_w)
    args = _mrope_args(T, D, pos_thw, inv_freq, sections, norm_w, eps, cycled, interleaved)

    def half(x, out, name):
        if x is None:
            return None, 0, 0, 0
        H = _shape3(x, name)[1]
        xs = _rows3(x, name, T, H, D)
        if out is None:
            return _new(x, (T, H, D), _BF16, stream), H, xs, H * D
        return out, H, xs, _rows3(out, name + "_out", T, H, D)

    q_out, Hq, qs, qos = half(q, q_out, "q")
    k_out, Hk, ks, kos = half(k, k_out, "k")
    _call("vit_qk_norm_mrope", dev, stream, _addr(q), _addr(q_out), _addr(k), _addr(k_out), T, Hq, Hk, D, qs, qos, ks,
          kos, *args)
    return q_out, k_out


def qk_norm_mrope_bwd(dq: torch.Tensor | None, dk: torch.Tensor | None, q: torch.Tensor | None,
                      k: torch.Tensor | None, pos_thw: torch.Tensor, inv_freq: torch.Tensor, sections,
                      norm_w: torch.Tensor | None = None, eps: float = 1e-6, *, cycled: bool = False,
                      interleaved: bool = False, inplace: bool = False, workspace: torch.Tensor | None = None,
                      stream=None):
    """Gradient of qk_norm_mrope: from dq, dk (with respect to its outputs; either may be None) and its inputs
    q, k (needed with norm_w only) returns (dq_in, dk_in, dnorm_w [2, D] fp32 or None). ``inplace`` writes
    over dq and dk."""
    ref = dq if dq is not None else dk
    if ref is None:
        raise ValueError("at least one of dq and dk is required")
    T, _, D = _shape3(ref, "dq and dk")
    dev = _device(dq, dk, q, k, pos_thw, inv_freq, norm_w, workspace)
    args = _mrope_args(T, D, pos_thw, inv_freq, sections, norm_w, eps, cycled, interleaved)

    def half(d, x, name):
        if d is None:
            return None, 0, 0, 0, 0, None
        H = _shape3(d, "d" + name)[1]
        ds, xs = _rows3(d, "d" + name, T, H, D), 0
        if norm_w is not None:
            if x is None:
                raise ValueError(f"{name} is needed for the gradient of its norm")
            xs = _rows3(x, name, T, H, D)
        else:
            x = None
        if inplace:
            return d, H, ds, ds, xs, x
        return _new(d, (T, H, D), _BF16, stream), H, ds, H * D, xs, x

    dq_in, Hq, dqs, dqis, qs, q = half(dq, q, "q")
    dk_in, Hk, dks, dkis, ks, k = half(dk, k, "k")
    dw = None
    if norm_w is not None:
        dw = _new(inv_freq, (2, D), _F32, stream)
        if workspace is None:
            workspace = _scratch(_size("vit_qk_norm_mrope_bwd_workspace_size", D), ref, stream)
    _call("vit_qk_norm_mrope_bwd", dev, stream, _addr(dq), _addr(dq_in), _addr(dk), _addr(dk_in), _addr(q), _addr(k),
          T, Hq, Hk, D, dqs, dqis, dks, dkis, qs, ks, *args, _addr(dw), _addr(workspace), _bytes(workspace))
    return dq_in, dk_in, dw


def _bytes(t: torch.Tensor | None) -> int:
    if t is None:
        return 0
    if not t.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return t.numel() * t.element_size()


def _word(status: torch.Tensor | None):
    """Address of a status word."""
    if status is None:
        return None
    if status.dtype is not _I32 or status.numel() < 1:
        raise ValueError("status must be a CUDA int32 tensor (new_status)")
    return status.data_ptr()


@functools.lru_cache(maxsize=256)
def _size(fn: str, *sizes) -> int:
    """Bytes of a workspace, a function of the sizes alone."""
    return getattr(lib(), fn)(*sizes)


def cross_attn_workspace_size(Tq: int, Tk: int, Hq: int, Hkv: int, D: int, B: int, max_q: int = 0,
                              max_k: int = 0) -> int:
    return int(lib().vit_cross_attn_workspace_size(int(Tq), int(Tk), *_ints(Hq, Hkv, D, B, max_q, max_k)))


def cross_attn_bwd_workspace_size(Tq: int, Tk: int, Hq: int, Hkv: int, D: int, B: int, max_q: int = 0,
                                  max_k: int = 0) -> int:
    return int(lib().vit_cross_attn_bwd_workspace_size(int(Tq), int(Tk), *_ints(Hq, Hkv, D, B, max_q, max_k)))


def _cross_lists(cu_q, cu_k, k_len) -> int:
    for name, t in (("cu_q", cu_q), ("cu_k", cu_k), ("k_len", k_len)):
        if t is not None and (t.dtype is not _I32 or t.dim() != 1 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA int32 vector")
    B = cu_q.numel() - 1
    if B < 0 or cu_k.numel() != B + 1 or (k_len is not None and k_len.numel() != B):
        raise ValueError("cu_q and cu_k must be [B + 1] and k_len [B]")
    return B


def _lse_ok(lse, T, H):
    if lse.dtype is not _F32 or tuple(lse.shape) != (T, H) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous CUDA float32 tensor [{T}, {H}]")


def cross_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
               max_q: int | None = None, max_k: int | None = None, scale: float | None = None, *,
               k_len: torch.Tensor | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, return_lse: bool = False,
               lse: torch.Tensor | None = None, stream=None):
    """Attention of packed queries q [Tq, Hq, D] over packed states k, v [Tk, Hkv, D] of other lengths, sequence
    by sequence (cu_q, cu_k [B + 1]; k_len [B]: real states per sequence where they are padded), without a causal
    mask; Hq is a multiple of Hkv. Serves prompts, single new tokens and latent queries. A sequence without
    states gets zeros and lse = -inf; rows of no sequence are left as they were (in tensors the call allocates: with
    any values). ``max_q`` and ``max_k`` bound the lengths (None: Tq, Tk); tight bounds are faster. With
    ``return_lse`` (or an ``lse`` buffer) returns (out, lse [Tq, Hq] fp32)."""
    Tq, Hq, D = _shape3(q, "q")
    Tk, Hkv, _ = _shape3(k, "k")
    dev = _device(q, k, v, cu_q, cu_k, k_len, out, workspace, status, lse)
    qs, ks, vs = _rows3(q, "q", Tq, Hq, D), _rows3(k, "k", Tk, Hkv, D), _rows3(v, "v", Tk, Hkv, D)
    B = _cross_lists(cu_q, cu_k, k_len)
    max_q, max_k = _max_seqlen(max_q), _max_seqlen(max_k)
    if out is None:
        out = _new(q, (Tq, Hq, D), _BF16, stream)
        os_ = Hq * D
    else:
        os_ = _rows3(out, "out", Tq, Hq, D)
    if lse is not None:
        _lse_ok(lse, Tq, Hq)
    elif return_lse:
        lse = _new(q, (Tq, Hq), _F32, stream)
    if workspace is None:
        workspace = _scratch(_size("vit_cross_attn_workspace_size", Tq, Tk, Hq, Hkv, D, B, max_q, max_k), q, stream)
    _call("vit_cross_attn", dev, stream, _addr(q), _addr(k), _addr(v), Tq, Tk, Hq, Hkv, D, qs, ks, vs, _addr(cu_q),
          _addr(cu_k), _addr(k_len), B, max_q, max_k, 0.0 if scale is None else float(scale), _addr(out), os_,
          _addr(lse), _addr(workspace), _bytes(workspace), _word(status))
    return (out, lse) if lse is not None else out


def cross_attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                   lse: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, max_q: int | None = None,
                   max_k: int | None = None, scale: float | None = None, *, k_len: torch.Tensor | None = None,
                   dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """Gradient of cross_attn: from dout and the forward call's inputs and results returns (dq, dk, dv), dk and dv
    summed over the query heads that share a key head. Rows of no sequence are 0 in the tensors the call
    allocates and left as they were in dq, dk, dv buffers it is given."""
    return _attn_bwd("vit_cross_attn_bwd", (), dout, q, k, v, out, lse, cu_q, cu_k, max_q, max_k, scale, k_len, dq, dk,
                     dv, workspace, status, stream)


def _attn_bwd(fn, mask, dout, q, k, v, out, lse, cu_q, cu_k, max_q, max_k, scale, k_len, dq, dk, dv, workspace, status,
              stream):
    Tq, Hq, D = _shape3(q, "q")
    Tk, Hkv, _ = _shape3(k, "k")
    dev = _device(dout, q, k, v, out, lse, cu_q, cu_k, k_len, dq, dk, dv, workspace, status)
    qs, ks, vs = _rows3(q, "q", Tq, Hq, D), _rows3(k, "k", Tk, Hkv, D), _rows3(v, "v", Tk, Hkv, D)
    dos, os_ = _rows3(dout, "dout", Tq, Hq, D), _rows3(out, "out", Tq, Hq, D)
    _lse_ok(lse, Tq, Hq)
    B = _cross_lists(cu_q, cu_k, k_len)
    max_q, max_k = _max_seqlen(max_q), _max_seqlen(max_k)
    given = [t is not None for t in (dq, dk, dv)]
    if any(given) and not all(given):
        raise ValueError("give all of dq, dk and dv, or none")
    if not any(given):
        dq, dk, dv = (_new(q, n, _BF16, stream) for n in ((Tq, Hq, D), (Tk, Hkv, D), (Tk, Hkv, D)))
    dqs, dks, dvs = _rows3(dq, "dq", Tq, Hq, D), _rows3(dk, "dk", Tk, Hkv, D), _rows3(dv, "dv", Tk, Hkv, D)
    if workspace is None:
        workspace = _scratch(_size(fn + "_workspace_size", Tq, Tk, Hq, Hkv, D, B, max_q, max_k, *mask), q, stream)
    _call(fn, dev, stream, _addr(dout), _addr(q), _addr(k), _addr(v), _addr(out), _addr(lse), Tq,
          Tk, Hq, Hkv, D, dos, qs, ks, vs, os_, _addr(cu_q), _addr(cu_k), _addr(k_len), B, max_q, max_k,
          *mask, 0.0 if scale is None else float(scale), _addr(dq), _addr(dk), _addr(dv), dqs, dks, dvs,
          0 if given[0] else 1, _addr(workspace), _bytes(workspace), _word(status))
    if B == 0 and not given[0]:                        # the library does nothing at all without sequences
        with torch.cuda.stream(stream):
            for t in (dq, dk, dv):
                t.zero_()
    return dq, dk, dv


def window_attn_workspace_size(Tq: int, Tk: int, Hq: int, Hkv: int, D: int, B: int, max_q: int = 0, max_k: int = 0,
                               window: int = 0, sinks: int = 0) -> int:
    return int(lib().vit_window_attn_workspace_size(int(Tq), int(Tk), *_ints(Hq, Hkv, D, B, max_q, max_k, window, sinks)))


def window_attn_bwd_workspace_size(Tq: int, Tk: int, Hq: int, Hkv: int, D: int, B: int, max_q: int = 0,
                                   max_k: int = 0, window: int = 0, sinks: int = 0) -> int:
    return int(lib().vit_window_attn_bwd_workspace_size(int(Tq), int(Tk),
                                                        *_ints(Hq, Hkv, D, B, max_q, max_k, window, sinks)))


def prefix_attn_workspace_size(Tq: int, Tp: int, Tk: int, Hq: int, Hkv: int, D: int, B: int, G: int, max_q: int = 0,
                               max_p: int = 0, max_k: int = 0) -> int:
    return int(lib().vit_prefix_attn_workspace_size(int(Tq), int(Tp), int(Tk),
                                                    *_ints(Hq, Hkv, D, B, G, max_q, max_p, max_k)))


def _window(window, sinks):
    """The C convention: 0 = no window."""
    w, s = (0 if window is None else int(window)), int(sinks)
    if (window is not None and w != window) or s != sinks:
        raise ValueError("window and sinks must be whole numbers")
    if window is not None and w < 1:
        raise ValueError("window must be at least 1, or None")
    return _c_int(w), _c_int(s)


def window_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                max_q: int | None = None, max_k: int | None = None, window: int | None = None, sinks: int = 0,
                scale: float | None = None, *, k_len: torch.Tensor | None = None, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, return_lse: bool = False,
                lse: torch.Tensor | None = None, stream=None):
    """Causal attention of packed sequences over their own tokens: the queries of a sequence, q [Tq, Hq, D], are the
    last ones of its keys k, v [Tk, Hkv, D] (cu_q, cu_k [B + 1]; k_len [B]: real rows per sequence where a cache is
    padded). A query at position p sees the keys j <= p with p - j < ``window`` (None: all of them) or j < ``sinks``.
    Serves prompts, continuations and single tokens over a cache. A query without a key to see (fewer keys than
    queries) gets zeros and lse = -inf; the rest is as for cross_attn."""
    Tq, Hq, D = _shape3(q, "q")
    Tk, Hkv, _ = _shape3(k, "k")
    dev = _device(q, k, v, cu_q, cu_k, k_len, out, workspace, status, lse)
    qs, ks, vs = _rows3(q, "q", Tq, Hq, D), _rows3(k, "k", Tk, Hkv, D), _rows3(v, "v", Tk, Hkv, D)
    B = _cross_lists(cu_q, cu_k, k_len)
    max_q, max_k = _max_seqlen(max_q), _max_seqlen(max_k)
    window, sinks = _window(window, sinks)
    if out is None:
        out = _new(q, (Tq, Hq, D), _BF16, stream)
        os_ = Hq * D
    else:
        os_ = _rows3(out, "out", Tq, Hq, D)
    if lse is not None:
        _lse_ok(lse, Tq, Hq)
    elif return_lse:
        lse = _new(q, (Tq, Hq), _F32, stream)
    if workspace is None:
        workspace = _scratch(_size("vit_window_attn_workspace_size", Tq, Tk, Hq, Hkv, D, B, max_q, max_k, window,
                                   sinks), q, stream)
    _call("vit_window_attn", dev, stream, _addr(q), _addr(k), _addr(v), Tq, Tk, Hq, Hkv, D, qs, ks, vs, _addr(cu_q),
          _addr(cu_k), _addr(k_len), B, max_q, max_k, window, sinks, 0.0 if scale is None else float(scale),
          _addr(out), os_, _addr(lse), _addr(workspace), _bytes(workspace), _word(status))
    return (out, lse) if lse is not None else out


def window_attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                    lse: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, max_q: int | None = None,
                    max_k: int | None = None, window: int | None = None, sinks: int = 0, scale: float | None = None, *,
                    k_len: torch.Tensor | None = None, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                    dv: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, stream=None):
    """Gradient of window_attn: from dout and the forward call's inputs and results returns (dq, dk, dv), dk and dv
    summed over the query heads that share a key head. Keys that no query sees and queries that see no key, or one,
    get 0; rows of no sequence are as in cross_attn_bwd."""
    window, sinks = _window(window, sinks)
    return _attn_bwd("vit_window_attn_bwd", (window, sinks), dout, q, k, v, out, lse, cu_q, cu_k, max_q, max_k, scale,
                     k_len, dq, dk, dv, workspace, status, stream)


def prefix_attn(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                cu_q: torch.Tensor, cu_prefix: torch.Tensor, cu_k: torch.Tensor, cu_group: torch.Tensor | None = None,
                max_q: int | None = None, max_prefix: int | None = None, max_k: int | None = None,
                scale: float | None = None, *, k_len: torch.Tensor | None = None, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, return_lse: bool = False,
                lse: torch.Tensor | None = None, stream=None):
    """Attention of sequences that share prefixes: the sequences cu_group[g] .. cu_group[g + 1] (None: all of them)
    see the rows cu_prefix[g] .. cu_prefix[g + 1] of k_prefix, v_prefix [Tp, Hkv, D] and behind them their own keys
    k, v [Tk, Hkv, D] causally, as in window_attn without a window. The prefix is read once for all of a group's
    short sequences. ``max_q``, ``max_prefix`` and ``max_k`` bound the lengths (None: Tq, Tp, Tk). The rest is
    as for window_attn."""
    Tq, Hq, D = _shape3(q, "q")
    Tk, Hkv, _ = _shape3(k, "k")
    Tp = _shape3(k_prefix, "k_prefix")[0]
    dev = _device(q, k_prefix, v_prefix, k, v, cu_q, cu_prefix, cu_k, cu_group, k_len, out, workspace, status, lse)
    qs, ks, vs = _rows3(q, "q", Tq, Hq, D), _rows3(k, "k", Tk, Hkv, D), _rows3(v, "v", Tk, Hkv, D)
    kps, vps = _rows3(k_prefix, "k_prefix", Tp, Hkv, D), _rows3(v_prefix, "v_prefix", Tp, Hkv, D)
    B = _cross_lists(cu_q, cu_k, k_len)
    for name, t in (("cu_prefix", cu_prefix), ("cu_group", cu_group)):
        if t is not None and (t.dtype is not _I32 or t.dim() != 1 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA int32 vector")
    G = cu_prefix.numel() - 1
    if G < 0 or (cu_group is None and G != 1) or (cu_group is not None and cu_group.numel() != G + 1):
        raise ValueError("cu_prefix and cu_group must be [G + 1], G = 1 without cu_group")
    max_q, max_p, max_k = _max_seqlen(max_q), _max_seqlen(max_prefix), _max_seqlen(max_k)
    if out is None:
        out = _new(q, (Tq, Hq, D), _BF16, stream)
        os_ = Hq * D
    else:
        os_ = _rows3(out, "out", Tq, Hq, D)
    if lse is not None:
        _lse_ok(lse, Tq, Hq)
    elif return_lse:
        lse = _new(q, (Tq, Hq), _F32, stream)
    if workspace is None:
        workspace = _scratch(_size("vit_prefix_attn_workspace_size", Tq, Tp, Tk, Hq, Hkv, D, B, G, max_q, max_p,
                                   max_k), q, stream)
    _call("vit_prefix_attn", dev, stream, _addr(q), _addr(k_prefix), _addr(v_prefix), _addr(k), _addr(v), Tq, Tp, Tk,
          Hq, Hkv, D, qs, kps, vps, ks, vs, _addr(cu_q), _addr(cu_group), _addr(cu_prefix), _addr(cu_k), _addr(k_len),
          B, G, max_q, max_p, max_k, 0.0 if scale is None else float(scale), _addr(out), os_, _addr(lse),
          _addr(workspace), _bytes(workspace), _word(status))
    return (out, lse) if lse is not None else out


RES_BF16, RES_FP32 = 0, 1


def _rows2(t: torch.Tensor, name: str, T: int, C: int, dtype) -> int:
    """Row stride of [T, C] with unit element stride."""
    if t.shape != (T, C):
        raise ValueError(f"{name} must be [{T}, {C}], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    st = t.stride()
    if st[1] != 1 and C > 1:
        raise ValueError(f"{name} needs unit element stride (got strides {st})")
    return st[0] if T > 1 else C


def _channel(t: torch.Tensor | None, name: str, C: int):
    if t is not None and (t.dtype is not _BF16 or t.shape != (C,) or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor [{C}]")


def _residual(x: torch.Tensor):
    if x.dim() != 2 or x.dtype not in (_BF16, _F32):
        raise ValueError("the residual must be a CUDA bfloat16 or float32 tensor [T, C]")
    T, C = x.shape
    return T, C, RES_FP32 if x.dtype is _F32 else RES_BF16


def _gate_stride(gate, T, C) -> int:
    if gate is None:
        return 0
    if gate.dim() == 1:
        _channel(gate, "gate", C)
        return 0
    stride = _rows2(gate, "gate", T, C, _BF16)
    if stride == 0:                                    # an expanded row: its gradient would be a [C] one
        raise ValueError("a gate for all tokens is given as [C]")
    return stride


def norm_residual(x: torch.Tensor, y: torch.Tensor, *, gate: torch.Tensor | None = None,
                  w_post: torch.Tensor | None = None, w_pre: torch.Tensor | None = None, scale: float = 1.0,
                  eps: float = 1e-6, h_out: torch.Tensor | None = None, z_out: torch.Tensor | None = None,
                  stream=None):
    """h = x + scale * gate * RMSNorm(y; w_post); z = RMSNorm(h; w_pre). Returns (h, z), z None without w_pre.

    x [T, C] bf16 or fp32 (h has its type and may be x itself), y [T, C] bf16 (z may be y itself), gate [C] or
    [T, C] bf16, the weights [C] bf16. Without w_post y is taken as it is."""
    T, C, res = _residual(x)
    dev = _device(x, y, gate, w_post, w_pre, h_out, z_out)
    xs, ys = _rows2(x, "x", T, C, x.dtype), _rows2(y, "y", T, C, _BF16)
    gs = _gate_stride(gate, T, C)
    _channel(w_post, "w_post", C)
    _channel(w_pre, "w_pre", C)
    if w_pre is None and z_out is not None:
        raise ValueError("z_out needs w_pre")
    hs = zs = C
    if h_out is None:
        h_out = _new(x, (T, C), x.dtype, stream)
    else:
        hs = _rows2(h_out, "h_out", T, C, x.dtype)
    if z_out is not None:
        zs = _rows2(z_out, "z_out", T, C, _BF16)
    elif w_pre is not None:
        z_out = _new(y, (T, C), _BF16, stream)
    _call("vit_norm_residual", dev, stream, _addr(x), _addr(y), _addr(gate), _addr(w_post), _addr(w_pre),
          _addr(h_out), _addr(z_out), T, C, res, xs, ys, gs, hs, zs, float(scale), float(eps))
    return h_out, z_out


def norm_residual_bwd(dz: torch.Tensor | None, dh: torch.Tensor | None, h: torch.Tensor | None,
                      y: torch.Tensor | None, *, gate: torch.Tensor | None = None,
                      w_post: torch.Tensor | None = None, w_pre: torch.Tensor | None = None, scale: float = 1.0,
                      eps: float = 1e-6, workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      stream=None):
    """Gradient of norm_residual: from dz (given exactly when w_pre is), dh (the residual stream's own gradient,
    or None), the stored h (needed with w_pre) and y (needed with w_post or gate) returns (dx, dy, dgate, dw_post,
    dw_pre); the last three are None without gate, w_post, w_pre. dgate is fp32 [C] for a [C] gate and bf16 [T, C]
    for a [T, C] one."""
    ref = dh if dh is not None else h
    if ref is None:
        raise ValueError("dh or h is required")
    if (dz is None) != (w_pre is None):
        raise ValueError("dz is given exactly when w_pre is")
    if w_pre is not None and h is None:
        raise ValueError("h is needed for the gradient of the norm after the residual")
    if dz is None and dh is None:
        raise ValueError("at least one of dz and dh is required")
    if y is None and (w_post is not None or gate is not None):
        raise ValueError("y is needed for the gradient of its norm or gate")
    T, C, res = _residual(ref)
    dev = _device(dz, dh, h, y, gate, w_post, w_pre, workspace, status)
    ds = _rows2(dh, "dh", T, C, ref.dtype) if dh is not None else 0
    zs = _rows2(dz, "dz", T, C, _BF16) if dz is not None else 0
    hs = _rows2(h, "h", T, C, ref.dtype) if h is not None else 0
    ys = _rows2(y, "y", T, C, _BF16) if y is not None else 0
    gs = _gate_stride(gate, T, C)
    _channel(w_post, "w_post", C)
    _channel(w_pre, "w_pre", C)
    dx, dy = _new(ref, (T, C), ref.dtype, stream), _new(ref, (T, C), _BF16, stream)
    whole = gate is not None and gate.dim() == 1       # one gate for all tokens
    dgate = None if gate is None else _new(ref, (C,), _F32, stream) if whole else _new(ref, (T, C), _BF16, stream)
    dw_post = None if w_post is None else _new(ref, (C,), _F32, stream)
    dw_pre = None if w_pre is None else _new(ref, (C,), _F32, stream)
    sums = whole or w_post is not None or w_pre is not None
    if workspace is None:
        workspace = _scratch(_size("vit_norm_residual_bwd_workspace_size", C) if sums else 0, ref, stream)
    _call("vit_norm_residual_bwd", dev, stream, _addr(dz), _addr(dh), _addr(h), _addr(y), _addr(gate), _addr(w_post),
          _addr(w_pre), _addr(dx), _addr(dy), _addr(dgate), _addr(dw_post), _addr(dw_pre), T, C, res, zs, ds, hs, ys,
          gs, C, C, C, float(scale), float(eps), _addr(workspace), _bytes(workspace), _word(status))
    return dx, dy, dgate, dw_post, dw_pre


DEFAULT_SHORT_MAX = 64   # the library's kernel split when a call passes none


def launch_count() -> int:
    return int(lib().vit_launch_count())


def kernel_timing(enable: bool) -> bool:
    return bool(lib().vit_kernel_timing(1 if enable else 0))


def kernel_timing_read(max_entries: int = 32) -> dict:
    """{kernel name: (launches, total ms)} for launches timed since the last read (synchronises)."""
    arr = (_KernelTime * max_entries)()
    n = lib().vit_kernel_timing_read(arr, max_entries)
    if n < 0:
        raise VitError(-8, "vit_kernel_timing_read")
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms)) for i in range(n)}


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
