"""Thin ctypes binding over libmxqdq.so (argument marshalling only).

Every function has the name of the C entry point it calls and takes torch
tensors on the GPU.  Before anything is enqueued it checks every tensor it
is handed: dtype and exact shape first (codes [M, K/2] or [M, K], scales
[M, K/32] or [M, K/16] for NVFP4, blocked scales at least the blocked size,
outputs [M, K] in the stated dtype), then that each is a contiguous tensor
on the current device; a mismatch raises ValueError or TypeError.  It then points the
library at torch's current stream and passes raw pointers.  All computation
happens in the HIP kernels; there is no fallback: if the library is missing
the import fails.  Nothing is recorded for autograd, except by mx_rope.

Tensor conventions: bf16 data is ``torch.bfloat16``; codes and scales are
``torch.uint8``; the rotation is an r x r tensor in the source dtype.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("LIBMXQDQ", os.path.join(_HERE, "libmxqdq.so"))

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libmxqdq.so not found at {LIB_PATH}; build it with "
                      "`python -m microscaling_quantize_dequantize_amd.build`")

_lib = ctypes.CDLL(LIB_PATH)

E2M1, E4M3 = 0, 1
BF16, F32 = 0, 1
ROWMAJOR, BLOCKED = 0, 1
HALF, INTERLEAVED = 0, 1
ATTENTION_DIMS = (64, 96, 128, 192, 256)
_DTYPE = {torch.bfloat16: BF16, torch.float32: F32}

_vp, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_lib.mx_qdq.argtypes = [_int, _vp, _int, _i64, _i64, _vp, _int, _vp]
_lib.mx_quantize.argtypes = [_int, _vp, _i64, _i64, _vp, _int, _vp, _vp]
_lib.mx_dequantize.argtypes = [_int, _vp, _vp, _i64, _i64, _int, _vp]
_lib.mx_rotate.argtypes = [_vp, _int, _i64, _i64, _vp, _int, _vp]
_lib.mx_matmul.argtypes = [_int, _vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, ctypes.c_float, _int, _vp]
_lib.mx_blocked_scales_bytes.argtypes = [_i64, _i64]
_lib.mx_blocked_scales_bytes.restype = _i64
_lib.mx_scales_to_blocked.argtypes = [_vp, _i64, _i64, _vp]
_lib.mx_quantize_blocked.argtypes = [_int, _vp, _i64, _i64, _vp, _int, _vp, _vp]
_lib.mx_nvfp4_quantize.argtypes = [_vp, _i64, _i64, _vp, _int, _vp, _vp, _vp]
_lib.mx_nvfp4_qdq.argtypes = [_vp, _i64, _i64, _vp, _int, _vp, _vp]
_lib.mx_nvfp4_dequantize.argtypes = [_vp, _vp, _i64, _i64, _vp, _int, _vp]
_dbl = ctypes.c_double
_lib.mx_rope.argtypes = [_vp, _i64, _i64, _int, _i64, _i64, _i64, _vp, _vp, _i64, _int, _dbl, _int, _vp, _i64, _i64]
_lib.mx_cache_write.argtypes = [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _int, _dbl]
_lib.mx_cache_read.argtypes = [_vp, _vp, _i64, _vp, _vp]
_lib.mx_cache_attention_workspace.argtypes = [_vp, _i64, _i64, _i64, _i64, _i64]
_lib.mx_cache_attention_workspace.restype = _i64
_lib.mx_cache_attention.argtypes = [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp,
                                    _i64, ctypes.c_float, _vp, _vp, _i64]
_lib.mx_set_stream.argtypes = [_vp]
_lib.mx_set_stream.restype = None
_lib.mx_get_stream.restype = _vp
_lib.mx_status_string.argtypes = [_int]
_lib.mx_status_string.restype = ctypes.c_char_p
for _f in (_lib.mx_qdq, _lib.mx_quantize, _lib.mx_dequantize, _lib.mx_rotate, _lib.mx_matmul,
           _lib.mx_scales_to_blocked, _lib.mx_quantize_blocked, _lib.mx_nvfp4_quantize, _lib.mx_nvfp4_qdq,
           _lib.mx_nvfp4_dequantize, _lib.mx_rope, _lib.mx_cache_write, _lib.mx_cache_read,
           _lib.mx_cache_attention):
    _f.restype = _int


class MXError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(f"libmxqdq status {status}: {mx_status_string(status)}")


def mx_status_string(status: int) -> str:
    return _lib.mx_status_string(int(status)).decode()


def mx_set_stream(stream) -> None:
    """Point the calling thread's library calls at a torch stream or a raw
    hipStream_t (int)."""
    _lib.mx_set_stream(ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream))


def _dev(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if t.device.index != torch.cuda.current_device():
        # the library launches on the current device (and torch's stream there)
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _want(t, name: str, dtype: torch.dtype, shape) -> None:
    """t must be a tensor of exactly this dtype and shape (checked before any
    pointer is taken, so that a wrong buffer never reaches a kernel)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _want_blocked(t, name: str, M: int, K: int) -> None:
    """Blocked scales: a flat uint8 tensor of at least the blocked size."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != torch.uint8 or t.dim() != 1:
        raise ValueError(f"{name} must be a flat uint8 tensor")
    need = mx_blocked_scales_bytes(M, K)
    if t.numel() < need:
        raise ValueError(f"{name} holds {t.numel()} bytes; the blocked layout of {M} x {K} needs {need}")


def _rot(rot, dtype):
    if rot is None:
        return None, 0
    if not isinstance(rot, torch.Tensor) or rot.dtype != dtype or rot.dim() != 2 or rot.shape[0] != rot.shape[1]:
        raise ValueError("rotation must be a square matrix in the source dtype")
    return _dev(rot, "rot"), rot.shape[0]


def _mk(src: torch.Tensor) -> tuple[int, int]:
    if not isinstance(src, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if src.dim() != 2:
        raise ValueError("expected a 2-D [M, K] tensor")
    return src.shape[0], src.shape[1]


def _code_cols(fmt: int, K: int) -> int:
    return K // 2 if fmt == E2M1 else K


def _call(status: int) -> None:
    if status != 0:
        raise MXError(status)


# The handle of a device's current stream: the public call builds a Stream object around it, 3 us of a call's 10, so the
# one that torch's own compiled code takes is used where there is one.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream() -> None:
    _lib.mx_set_stream(_current_stream(torch.cuda.current_device()))


def mx_qdq(fmt: int, src: torch.Tensor, rot: torch.Tensor | None = None,
           dst: torch.Tensor | None = None) -> torch.Tensor:
    """Fused MX quantize-dequantize of src [M, K] (bf16 or fp32) into dst."""
    M, K = _mk(src)
    if src.dtype not in _DTYPE:
        raise TypeError("src must be bfloat16 or float32")
    if dst is None:
        dst = torch.empty_like(src)
    _want(dst, "dst", src.dtype, (M, K))
    ps, pd = _dev(src, "src"), _dev(dst, "dst")
    rp, r = _rot(rot, src.dtype)
    _stream()
    _call(_lib.mx_qdq(fmt, ps, _DTYPE[src.dtype], M, K, rp, r, pd))
    return dst


def mx_quantize(fmt: int, src: torch.Tensor, rot: torch.Tensor | None = None,
                codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """Quantize bf16 src [M, K] -> (codes uint8 [M, K/2 or K], scales uint8 [M, K/32])."""
    M, K = _mk(src)
    if src.dtype != torch.bfloat16:
        raise TypeError("mx_quantize takes bfloat16 input")
    if codes is None:
        codes = torch.empty((M, _code_cols(fmt, K)), dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = torch.empty((M, K // 32), dtype=torch.uint8, device=src.device)
    _want(codes, "codes", torch.uint8, (M, _code_cols(fmt, K)))
    _want(scales, "scales", torch.uint8, (M, K // 32))
    ps, pc, pq = _dev(src, "src"), _dev(codes, "codes"), _dev(scales, "scales")
    rp, r = _rot(rot, src.dtype)
    _stream()
    _call(_lib.mx_quantize(fmt, ps, M, K, rp, r, pc, pq))
    return codes, scales


def mx_dequantize(fmt: int, codes: torch.Tensor, scales: torch.Tensor, K: int,
                  dtype: torch.dtype = torch.bfloat16, dst: torch.Tensor | None = None):
    """Dequantize codes [M, K/2 or K] + row-major scales [M, K/32] into a
    [M, K] tensor of `dtype`."""
    if not isinstance(scales, torch.Tensor) or scales.dim() != 2:
        raise ValueError("scales must be a 2-D [M, K/32] uint8 tensor")
    M = scales.shape[0]
    _want(scales, "scales", torch.uint8, (M, K // 32))
    _want(codes, "codes", torch.uint8, (M, _code_cols(fmt, K)))
    if dst is None:
        dst = torch.empty((M, K), dtype=dtype, device=codes.device)
    if dst.dtype not in _DTYPE:
        raise ValueError("dst must be bfloat16 or float32")
    _want(dst, "dst", dst.dtype, (M, K))
    pc, pq, pd = _dev(codes, "codes"), _dev(scales, "scales"), _dev(dst, "dst")
    _stream()
    _call(_lib.mx_dequantize(fmt, pc, pq, M, K, _DTYPE[dst.dtype], pd))
    return dst


def mx_rotate(src: torch.Tensor, rot: torch.Tensor, dst: torch.Tensor | None = None):
    """The rotation step alone: fp32 [M, K] of per-chunk src . rot."""
    M, K = _mk(src)
    if src.dtype not in _DTYPE:
        raise TypeError("src must be bfloat16 or float32")
    if dst is None:
        dst = torch.empty((M, K), dtype=torch.float32, device=src.device)
    _want(dst, "dst", torch.float32, (M, K))
    ps, pd = _dev(src, "src"), _dev(dst, "dst")
    rp, r = _rot(rot, src.dtype)
    _stream()
    _call(_lib.mx_rotate(ps, _DTYPE[src.dtype], M, K, rp, r, pd))
    return dst


def mx_blocked_scales_bytes(M: int, K: int) -> int:
    n = _lib.mx_blocked_scales_bytes(M, K)
    if n < 0:
        raise MXError(n)
    return n


def mx_scales_to_blocked(scales: torch.Tensor, K: int, blocked: torch.Tensor | None = None) -> torch.Tensor:
    """Row-major [M, K/32] scales -> the blocked layout (flat uint8)."""
    if not isinstance(scales, torch.Tensor) or scales.dim() != 2:
        raise ValueError("scales must be a 2-D [M, K/32] uint8 tensor")
    M = scales.shape[0]
    _want(scales, "scales", torch.uint8, (M, K // 32))
    if blocked is None:
        blocked = torch.empty(mx_blocked_scales_bytes(M, K), dtype=torch.uint8, device=scales.device)
    _want_blocked(blocked, "blocked", M, K)
    pq, pb = _dev(scales, "scales"), _dev(blocked, "blocked")
    _stream()
    _call(_lib.mx_scales_to_blocked(pq, M, K, pb))
    return blocked


def mx_quantize_blocked(fmt: int, src: torch.Tensor, rot: torch.Tensor | None = None,
                        codes: torch.Tensor | None = None, blocked: torch.Tensor | None = None):
    """Quantize bf16 src [M, K] -> (codes, scales in the blocked layout)."""
    M, K = _mk(src)
    if src.dtype != torch.bfloat16:
        raise TypeError("mx_quantize_blocked takes bfloat16 input")
    if codes is None:
        codes = torch.empty((M, _code_cols(fmt, K)), dtype=torch.uint8, device=src.device)
    if blocked is None:
        blocked = torch.empty(mx_blocked_scales_bytes(M, K), dtype=torch.uint8, device=src.device)
    _want(codes, "codes", torch.uint8, (M, _code_cols(fmt, K)))
    _want_blocked(blocked, "blocked", M, K)
    ps, pc, pb = _dev(src, "src"), _dev(codes, "codes"), _dev(blocked, "blocked")
    rp, r = _rot(rot, src.dtype)
    _stream()
    _call(_lib.mx_quantize_blocked(fmt, ps, M, K, rp, r, pc, pb))
    return codes, blocked


def _want_scales(t, name: str, layout: int, rows: int, K: int) -> None:
    if layout == BLOCKED:
        _want_blocked(t, name, rows, K)
    else:
        _want(t, name, torch.uint8, (rows, K // 32))


def mx_matmul(fmt: int, a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
              b_scales: torch.Tensor, K: int, alpha: float = 1.0, dtype: torch.dtype = torch.bfloat16,
              c: torch.Tensor | None = None, scale_layout: int = ROWMAJOR):
    """[M, N] = alpha * A_dq . B_dq^T from MX codes and scales (A [M, K], B [N, K]);
    the row counts come from the codes."""
    for t, name in ((a_codes, "a_codes"), (b_codes, "b_codes")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D uint8 tensor")
    M, N = a_codes.shape[0], b_codes.shape[0]
    _want(a_codes, "a_codes", torch.uint8, (M, _code_cols(fmt, K)))
    _want(b_codes, "b_codes", torch.uint8, (N, _code_cols(fmt, K)))
    if scale_layout in (ROWMAJOR, BLOCKED):
        _want_scales(a_scales, "a_scales", scale_layout, M, K)
        _want_scales(b_scales, "b_scales", scale_layout, N, K)
    if c is None:
        c = torch.empty((M, N), dtype=dtype, device=a_codes.device)
    if not isinstance(c, torch.Tensor) or c.dtype not in _DTYPE or tuple(c.shape) != (M, N):
        raise ValueError("c must be a bfloat16 or float32 [M, N] tensor")
    pa, pas, pb, pbs, pc = (_dev(a_codes, "a_codes"), _dev(a_scales, "a_scales"), _dev(b_codes, "b_codes"),
                            _dev(b_scales, "b_scales"), _dev(c, "c"))
    _stream()
    _call(_lib.mx_matmul(fmt, pa, pas, pb, pbs, scale_layout, M, N, K, float(alpha), _DTYPE[c.dtype], pc))
    return c


def _want_g(global_scale) -> None:
    if not isinstance(global_scale, torch.Tensor) or global_scale.dtype != torch.float32 \
            or global_scale.numel() != 1:
        raise ValueError("global_scale must be a one-element float32 tensor")


def _gscale(global_scale: torch.Tensor) -> int:
    _want_g(global_scale)
    return _dev(global_scale, "global_scale")


def mx_nvfp4_quantize(src: torch.Tensor, global_scale: torch.Tensor, rot: torch.Tensor | None = None,
                      codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """NVFP4 quantize of bf16 src [M, K] -> (E2M1 codes [M, K/2], E4M3 scale bytes [M, K/16])."""
    M, K = _mk(src)
    if src.dtype != torch.bfloat16:
        raise TypeError("mx_nvfp4_quantize takes bfloat16 input")
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = torch.empty((M, K // 16), dtype=torch.uint8, device=src.device)
    _want(codes, "codes", torch.uint8, (M, K // 2))
    _want(scales, "scales", torch.uint8, (M, K // 16))
    _want_g(global_scale)
    ps, pc, pq, pg = _dev(src, "src"), _dev(codes, "codes"), _dev(scales, "scales"), _gscale(global_scale)
    rp, r = _rot(rot, src.dtype)
    _stream()
    _call(_lib.mx_nvfp4_quantize(ps, M, K, rp, r, pg, pc, pq))
    return codes, scales


def mx_nvfp4_qdq(src: torch.Tensor, global_scale: torch.Tensor, rot: torch.Tensor | None = None,
                 dst: torch.Tensor | None = None) -> torch.Tensor:
    """NVFP4 quantize-dequantize of bf16 src [M, K] into bf16 dst."""
    M, K = _mk(src)
    if src.dtype != torch.bfloat16:
        raise TypeError("mx_nvfp4_qdq takes bfloat16 input")
    if dst is None:
        dst = torch.empty_like(src)
    _want(dst, "dst", torch.bfloat16, (M, K))
    _want_g(global_scale)
    ps, pd, pg = _dev(src, "src"), _dev(dst, "dst"), _gscale(global_scale)
    rp, r = _rot(rot, src.dtype)
    _stream()
    _call(_lib.mx_nvfp4_qdq(ps, M, K, rp, r, pg, pd))
    return dst


def mx_nvfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, K: int, global_scale: torch.Tensor,
                        dtype: torch.dtype = torch.bfloat16, dst: torch.Tensor | None = None):
    """NVFP4 codes [M, K/2] + E4M3 scales [M, K/16] -> [M, K] of `dtype`."""
    if not isinstance(scales, torch.Tensor) or scales.dim() != 2:
        raise ValueError("scales must be a 2-D [M, K/16] uint8 tensor")
    M = scales.shape[0]
    _want(scales, "scales", torch.uint8, (M, K // 16))
    _want(codes, "codes", torch.uint8, (M, K // 2))
    if dst is None:
        dst = torch.empty((M, K), dtype=dtype, device=codes.device)
    if dst.dtype not in _DTYPE:
        raise ValueError("dst must be bfloat16 or float32")
    _want(dst, "dst", dst.dtype, (M, K))
    _want_g(global_scale)
    pc, pq, pd, pg = _dev(codes, "codes"), _dev(scales, "scales"), _dev(dst, "dst"), _gscale(global_scale)
    _stream()
    _call(_lib.mx_nvfp4_dequantize(pc, pq, M, K, pg, _DTYPE[dst.dtype], pd))
    return dst


# ---- rotary positions, the paged MX cache and attention over it ---------------


def _place(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _heads(t, name: str, dtypes, shape=None):
    """t must be [tokens, heads, dim] with contiguous dimensions (any token and head strides) on the current
    device.  Its pointer and the two strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {'[tokens, heads, dim]' if shape is None else tuple(shape)}, "
                         f"got {tuple(t.shape)}")
    token, head, one = t.stride()
    if one != 1 and t.shape[2] > 1:
        raise ValueError(f"the dimensions of {name} must be contiguous")
    _place(t, name)
    # the stride of a single token or head is whatever its view left there
    return t.data_ptr(), token if t.shape[0] > 1 else 0, head if t.shape[1] > 1 else 0


def _vector(t, name: str, dtype: torch.dtype, n: int) -> int:
    """Pointer of a contiguous [n] tensor of this type on the current device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype or t.shape != (n,):
        raise ValueError(f"{name} must be {dtype} [{n}], got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _place(t, name)
    return t.data_ptr()


def _rotary(positions, inv_freq, tokens: int):
    """Pointers of the positions and frequencies, and the number of rotated dimensions."""
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a one-dimensional float64 tensor (angle per position of each pair)")
    pairs = inv_freq.shape[0]
    return (_vector(positions, "positions", torch.int64, tokens), _vector(inv_freq, "inv_freq", torch.float64, pairs),
            2 * pairs)


def _like(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def mx_rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, layout: int = HALF, scale: float = 1.0,
            inverse: bool = False, dst: torch.Tensor | None = None) -> torch.Tensor:
    """Rotary positions on the first 2 * len(inv_freq) dimensions of x [tokens, heads, dim] (bf16 or fp32, any token
    and head strides), the others copied.

    positions int64 [tokens]; inv_freq float64 [pairs]; layout HALF (dimension p with p + pairs) or INTERLEAVED
    (2p with 2p + 1); scale multiplies the rotated dimensions.  inverse: the transposed rotation, which takes the
    gradient of the output to that of x.  dst may be x itself.  Without dst the call is recorded for autograd if x
    requires a gradient (inv_freq gets none); with dst nothing is recorded."""
    ps, st, sh = _heads(x, "x", (torch.bfloat16, torch.float32))
    if x.requires_grad and dst is None and torch.is_grad_enabled():
        return _Rope.apply(x, positions, inv_freq, layout, scale, inverse)
    tokens, heads, dim = x.shape
    if dst is None:  # what is allocated here needs no check
        dst = _like(x)
        pd, dt, dh = dst.data_ptr(), heads * dim, dim
    else:
        pd, dt, dh = _heads(dst, "dst", (x.dtype,), x.shape)
    pp, pf, rot = _rotary(positions, inv_freq, tokens)
    _stream()
    _call(_lib.mx_rope(ps, st, sh, _DTYPE[x.dtype], tokens, heads, dim, pp, pf, rot, layout, scale,
                       1 if inverse else 0, pd, dt, dh))
    return dst


class _Rope(torch.autograd.Function):
    """mx_rope with its gradient, the transposed rotation of that of the output (and the other way round)."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, layout, scale, inverse):
        ctx.save_for_backward(positions, inv_freq)
        ctx.rotation = layout, scale, inverse
        return mx_rope(x, positions, inv_freq, layout, scale, inverse)

    @staticmethod
    def backward(ctx, grad):
        layout, scale, inverse = ctx.rotation
        if grad.stride(2) != 1:  # that of a sum, say, is one value for all
            grad = grad.contiguous()
        return mx_rope(grad, *ctx.saved_tensors, layout, scale, not inverse), None, None, None, None, None


class _CacheStruct(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("heads", ctypes.c_int32), ("page", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("pages", _i64), ("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp)]


class MXCache:
    """A paged cache of keys and values in MX codes over the caller's tensors.

    fmt E2M1 or E4M3; codes uint8 [pages, heads, page, dim/2 or dim]; scales uint8 [pages, heads, dim/32, page].
    Token slots are page number * page + row.  The handle keeps the four tensors; it may be used on any stream.
    dim is a multiple of 32 up to 256; attention takes 64, 96, 128, 192 and 256 of these."""

    def __init__(self, fmt: int, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                 v_scales: torch.Tensor):
        if fmt not in (E2M1, E4M3):
            raise ValueError("fmt must be E2M1 or E4M3")
        if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4:
            raise ValueError("k_codes must be a 4-D uint8 tensor [pages, heads, page, dim/2 or dim]")
        pages, heads, page, cols = k_codes.shape
        if not 1 <= heads <= 65535:
            raise ValueError(f"a cache has 1 to 65535 heads, got {heads}")
        dim = 2 * cols if fmt == E2M1 else cols
        if dim % 32 or not 32 <= dim <= 256:
            raise ValueError(f"the head's dimension must be a multiple of 32 up to 256, got {dim}")
        if page < 16 or page > 65536 or page & (page - 1):
            raise ValueError(f"a page must hold a power of two of tokens, 16 at least, got {page}")
        _want(k_codes, "k_codes", torch.uint8, (pages, heads, page, cols))
        _want(v_codes, "v_codes", torch.uint8, (pages, heads, page, cols))
        _want(k_scales, "k_scales", torch.uint8, (pages, heads, dim // 32, page))
        _want(v_scales, "v_scales", torch.uint8, (pages, heads, dim // 32, page))
        ptrs = [_dev(t, n) for t, n in ((k_codes, "k_codes"), (k_scales, "k_scales"), (v_codes, "v_codes"),
                                        (v_scales, "v_scales"))]
        self.fmt, self.pages, self.heads, self.page, self.dim = fmt, pages, heads, page, dim
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.device = k_codes.device
        self._struct = _CacheStruct(fmt, heads, page, dim, pages, *ptrs)
        self._ref = ctypes.addressof(self._struct)
        self._bf16 = k_codes.new_empty(0, dtype=torch.bfloat16)  # new_empty of this is quicker than torch.empty

    @classmethod
    def allocate(cls, fmt: int, pages: int, heads: int, page: int, dim: int, device="cuda") -> "MXCache":
        """A cache of new tensors, all values zero."""
        cols = _code_cols(fmt, dim)

        def zeros(*shape):
            return torch.zeros(shape, dtype=torch.uint8, device=device)

        return cls(fmt, zeros(pages, heads, page, cols), zeros(pages, heads, dim // 32, page),
                   zeros(pages, heads, page, cols), zeros(pages, heads, dim // 32, page))


def _cache(cache) -> int:
    if not isinstance(cache, MXCache):
        raise TypeError("cache must be an MXCache")
    _place(cache.k_codes, "cache")
    return cache._ref


def mx_cache_write(cache: MXCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                   positions: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None, layout: int = HALF,
                   scale: float = 1.0) -> None:
    """Quantise keys and values [tokens, heads, dim] (bf16, any token and head strides) into the cache's slots
    (int64 [tokens]; slots outside the cache are skipped).  With positions and inv_freq the keys are rotated first, as
    by mx_rope, and rounded to bf16."""
    pc = _cache(cache)
    pk, kt, kh = _heads(k, "k", (torch.bfloat16,))
    shape = (k.shape[0], cache.heads, cache.dim)
    if k.shape != shape:
        raise ValueError(f"k must have shape {shape}, got {tuple(k.shape)}")
    pv, vt, vh = _heads(v, "v", (torch.bfloat16,), shape)
    ps = _vector(slots, "slots", torch.int64, shape[0])
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    pp, pf, rot = (None, None, 0) if positions is None else _rotary(positions, inv_freq, shape[0])
    _stream()
    _call(_lib.mx_cache_write(pc, pk, kt, kh, pv, vt, vh, ps, shape[0], pp, pf, rot, layout, scale))


def mx_cache_read(cache: MXCache, slots: torch.Tensor, k: torch.Tensor | None = None, v: torch.Tensor | None = None):
    """Keys and values of slots (int64 [tokens]) as bf16 [tokens, heads, dim]; zeros for slots outside the cache."""
    pc = _cache(cache)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a one-dimensional int64 tensor")
    shape = (slots.shape[0], cache.heads, cache.dim)
    for t, name in ((k, "k"), (v, "v")):
        if t is not None:
            _want(t, name, torch.bfloat16, shape)
            _dev(t, name)
    ps = _vector(slots, "slots", torch.int64, shape[0])
    if k is None:
        k = cache._bf16.new_empty(shape)
    if v is None:
        v = cache._bf16.new_empty(shape)
    pk, pv = k.data_ptr(), v.data_ptr()
    _stream()
    _call(_lib.mx_cache_read(pc, ps, shape[0], pk, pv))
    return k, v


def mx_cache_attention(cache: MXCache, q: torch.Tensor, q_starts: torch.Tensor, kv_lens: torch.Tensor,
                       block_table: torch.Tensor, max_q: int, max_kv: int, tree: torch.Tensor | None = None,
                       scale: float | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of new tokens over the cache: q [total_q, q_heads, dim] (bf16, any token and head strides that are
    multiples of 8) -> bf16 [total_q, q_heads, dim].

    Sequence b has the queries q_starts[b] .. q_starts[b + 1] (int32 [batch + 1]), and kv_lens[b] tokens (int32
    [batch]), of which the last are its new ones, one for each query; token t is in page block_table[b, t // page]
    (int32 [batch, pages of the longest], rows contiguous).  A query sees all tokens before the new ones, and of the
    new ones those up to its own, or with tree (int64 [total_q, words]) new token j where bit j % 64 of word j // 64 of
    its row is set.  A query that sees nothing gives zeros, and so does one of no sequence (from q_starts[batch] on).
    max_q, max_kv: at least the most queries and tokens of a sequence (with less, the rows of queries from max_q on are
    undefined and tokens from max_kv on are not seen).
    scale: dim ** -0.5 if not given."""
    pc = _cache(cache)
    pq, qt, qh = _heads(q, "q", (torch.bfloat16,))
    total, heads, dim = q.shape
    if dim != cache.dim or heads % cache.heads:
        raise ValueError(f"q must have {cache.dim} dimensions and a multiple of {cache.heads} heads, got "
                         f"{tuple(q.shape)}")
    if dim not in ATTENTION_DIMS:
        raise ValueError(f"attention takes heads of {', '.join(map(str, ATTENTION_DIMS))} dimensions, got {dim}")
    if not isinstance(kv_lens, torch.Tensor) or kv_lens.dim() != 1:
        raise ValueError("kv_lens must be a one-dimensional int32 tensor")
    batch = kv_lens.shape[0]
    pl = _vector(kv_lens, "kv_lens", torch.int32, batch)
    pst = _vector(q_starts, "q_starts", torch.int32, batch + 1)
    if not isinstance(block_table, torch.Tensor) or block_table.dtype != torch.int32 or block_table.dim() != 2 \
            or block_table.shape[0] != batch or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be an int32 tensor [batch, pages] with contiguous rows")
    _place(block_table, "block_table")
    pages = block_table.shape[1]
    stride = block_table.stride(0) if batch > 1 else pages
    pt, words = None, 0
    if tree is not None:
        if not isinstance(tree, torch.Tensor) or tree.dim() != 2:
            raise ValueError("tree must be an int64 tensor [total_q, words]")
        words = tree.shape[1]
        _want(tree, "tree", torch.int64, (total, words))
        if 64 * words < max_q:
            raise ValueError(f"tree has {words} words a row, max_q = {max_q} new tokens need {-(-max_q // 64)}")
        pt = _dev(tree, "tree")
    if out is None:
        out = _like(q)
    else:
        _want(out, "out", torch.bfloat16, (total, heads, dim))
        _dev(out, "out")
    po = out.data_ptr()
    need = _lib.mx_cache_attention_workspace(pc, heads, batch, total, max_q, max_kv)
    if need < 0:
        raise MXError(need)
    space = kv_lens.new_empty(need // 4) if need else None  # int32: 4 bytes each
    _stream()
    _call(_lib.mx_cache_attention(pc, pq, qt, qh, heads, pst, pl, batch, block_table.data_ptr(), stride, pages, total,
                                  max_q, max_kv, pt, words, dim ** -0.5 if scale is None else scale, po,
                                  space.data_ptr() if need else None, need))
    return out


def raw():
    """The ctypes library handle (for callers passing raw pointers)."""
    return _lib
