"""binary_bit_gemm_amd -- packed ternary / binary weight GEMM for AMD MI355X (gfx950).

Thin ctypes binding over liblowbit.so (include/lowbit.h).  Every step of the computation
runs in the library's HIP kernels; this module only checks tensor types, takes device
pointers and the current HIP stream, and raises on a non-zero status.  PyTorch is used for
device memory and streams only.

    import torch, binary_bit_gemm_amd as lb
    words, bad = lb.pack(codes_int8_cuda, bits=2)          # [N, K] -> [N, K/16] (int32 view)
    y = lb.gemm(x_bf16_cuda, words, scales_fp16_cuda, g=64, bits=2)
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import List, Optional, Sequence, Tuple

from ._lib import LowbitError, lib, library_path  # noqa: F401

TERNARY = 2
BINARY = 1
MAX_BATCH = 64


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream_ptr(device) -> int:
    torch = _torch()
    return int(torch.cuda.current_stream(device).cuda_stream)


def _check(status: int, what: str) -> None:
    if status != 0:
        L = lib()
        msg = L.lowbit_status_string(status).decode()
        hip = L.lowbit_last_hip_error()
        raise LowbitError(status, f"{what}: {msg}" + (f" (hipError {hip})" if status == 4 else ""))


def _require(t, dtype, name: str, ndim: int = 2):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def words_per_row(K: int, bits: int) -> int:
    return K * bits // 32


def pack(codes, bits: int, count_invalid: bool = True) -> Tuple["object", Optional[int]]:
    """int8 codes [N, K] on the GPU -> (packed words [N, K*bits/32] as int32, invalid count).

    The invalid count (codes outside {-1,0,1} / {-1,1}) is read back only when
    count_invalid is true (that synchronises the stream)."""
    torch = _torch()
    _require(codes, torch.int8, "codes")
    N, K = codes.shape
    words = torch.empty((N, words_per_row(K, bits)), dtype=torch.int32, device=codes.device)
    bad = torch.zeros(1, dtype=torch.int32, device=codes.device) if count_invalid else None
    st = lib().lowbit_pack(ctypes.c_void_p(codes.data_ptr()), ctypes.c_void_p(words.data_ptr()), N, K, bits,
                           ctypes.c_void_p(bad.data_ptr() if bad is not None else 0),
                           ctypes.c_void_p(_stream_ptr(codes.device)))
    _check(st, "lowbit_pack")
    return words, (int(bad.item()) if bad is not None else None)


def pack_u4(levels, count_invalid: bool = True):
    """Unsigned 4-bit levels (uint8 [N, K], 0 .. 15) on the GPU -> (packed words [N, K/8] as
    int32, invalid count) for lowbit_gemm_affine (lowbit_pack_u4)."""
    torch = _torch()
    _require(levels, torch.uint8, "levels")
    N, K = levels.shape
    words = torch.empty((N, K // 8), dtype=torch.int32, device=levels.device)
    bad = torch.zeros(1, dtype=torch.int32, device=levels.device) if count_invalid else None
    st = lib().lowbit_pack_u4(ctypes.c_void_p(levels.data_ptr()), ctypes.c_void_p(words.data_ptr()), N, K,
                              ctypes.c_void_p(bad.data_ptr() if bad is not None else 0),
                              ctypes.c_void_p(_stream_ptr(levels.device)))
    _check(st, "lowbit_pack_u4")
    return words, (int(bad.item()) if bad is not None else None)


def affine_workspace_size(M: int, N: int, K: int, g: int = 64) -> int:
    """Bytes of workspace lowbit_gemm_affine_ex can use for this shape (0: it takes no split)."""
    return int(lib().lowbit_affine_workspace_size(M, N, K, g))


def gemm_affine(x, words, scales, biases, g: int, out=None, workspace=None):
    """Y = X . W^T with affine 4-bit groups W = S * q + B (lowbit_gemm_affine): `words` from
    pack_u4, `scales` and `biases` fp16 [N, K/g].  `workspace`: an optional zero-filled device
    tensor of at least affine_workspace_size(M, N, K, g) bytes (lowbit_gemm_affine_ex), with which
    shapes whose tile grid leaves compute units idle split K across workgroups.  Up to 16 rows: gemv_affine is faster."""
    torch = _torch()
    _require(x, torch.bfloat16, "x")
    _require(words, torch.int32, "words")
    _require(scales, torch.float16, "scales")
    _require(biases, torch.float16, "biases")
    M, K = x.shape
    N = words.shape[0]
    if words.shape[1] != K // 8 or K % 8:
        raise ValueError(f"words must be [N, K/8] = [{N}, {K // 8}], got {tuple(words.shape)}")
    if K % g or tuple(scales.shape) != (N, K // g) or tuple(biases.shape) != (N, K // g):
        raise ValueError(f"scales and biases must be [N, K/g] = [{N}, {K // g if g else 0}]")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _require(out, torch.bfloat16, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N]")
    args = (ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(words.data_ptr()), ctypes.c_void_p(scales.data_ptr()),
            ctypes.c_void_p(biases.data_ptr()), ctypes.c_void_p(out.data_ptr()), M, N, K, g)
    if workspace is None:
        st = lib().lowbit_gemm_affine(*args, ctypes.c_void_p(_stream_ptr(x.device)))
        _check(st, "lowbit_gemm_affine")
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor")
        nbytes = workspace.numel() * workspace.element_size()
        st = lib().lowbit_gemm_affine_ex(*args, ctypes.c_void_p(workspace.data_ptr()), nbytes,
                                         ctypes.c_void_p(_stream_ptr(x.device)))
        _check(st, "lowbit_gemm_affine_ex")
    return out


def unpack(words, K: int, bits: int):
    """Packed words [N, K*bits/32] -> int8 codes [N, K]."""
    torch = _torch()
    _require(words, torch.int32, "words")
    N = words.shape[0]
    if words.shape[1] != words_per_row(K, bits):
        raise ValueError("words do not hold K codes per row")
    codes = torch.empty((N, K), dtype=torch.int8, device=words.device)
    st = lib().lowbit_unpack(ctypes.c_void_p(words.data_ptr()), ctypes.c_void_p(codes.data_ptr()), N, K, bits,
                             ctypes.c_void_p(_stream_ptr(words.device)))
    _check(st, "lowbit_unpack")
    return codes


LAYOUT_GEMLITE_U8T = 1  # uint8 [K/4, N]: GemLite's int2 weights, packed over K with a transpose
LAYOUT_MLX_U32 = 2      # uint32 [N, K/16]: MLX's packed rows


def _import(src, layout: int, N: int, K: int, zero: int, count_invalid: bool):
    torch = _torch()
    words = torch.empty((N, words_per_row(K, 2)), dtype=torch.int32, device=src.device)
    bad = torch.zeros(1, dtype=torch.int32, device=src.device) if count_invalid else None
    st = lib().lowbit_import_ternary(ctypes.c_void_p(src.data_ptr()), layout, zero, ctypes.c_void_p(words.data_ptr()),
                                     N, K, ctypes.c_void_p(bad.data_ptr() if bad is not None else 0),
                                     ctypes.c_void_p(_stream_ptr(src.device)))
    _check(st, "lowbit_import_ternary")
    return words, (int(bad.item()) if bad is not None else None)


def import_gemlite(src, N: int, K: int, zero: int = 1, count_invalid: bool = True):
    """GemLite int2 weights, uint8 [K/4, N] (transposed), levels q with code q - zero ->
    (packed words [N, K/16] as int32, invalid count).  N and K are the caller's: the
    orientation is never guessed from the buffer's shape, which is checked against them."""
    torch = _torch()
    _require(src, torch.uint8, "src")
    if tuple(src.shape) != (K // 4, N) or K % 4:
        raise ValueError(f"GemLite src must be uint8 [K/4, N] = ({K // 4}, {N}), got {tuple(src.shape)}")
    return _import(src, LAYOUT_GEMLITE_U8T, N, K, zero, count_invalid)


def import_mlx(src, N: int, K: int, zero: int = 1, count_invalid: bool = True):
    """MLX 2-bit rows, uint32 (or int32) [N, K/16], levels q with code q - zero -> (packed words
    [N, K/16] as int32, invalid count)."""
    torch = _torch()
    _require(src, torch.uint32 if src.dtype == torch.uint32 else torch.int32, "src")
    if tuple(src.shape) != (N, K // 16) or K % 16:
        raise ValueError(f"MLX src must be [N, K/16] = ({N}, {K // 16}), got {tuple(src.shape)}")
    return _import(src, LAYOUT_MLX_U32, N, K, zero, count_invalid)


def import_gemlite_binary(src, N: int, K: int):
    """GemLite 1-bit weights, uint8 [K/8, N] (transposed, bit i of byte (j, n) = code 8j + i,
    1 -> +1) -> packed binary words [N, K/32] as int32."""
    torch = _torch()
    _require(src, torch.uint8, "src")
    if tuple(src.shape) != (K // 8, N) or K % 8:
        raise ValueError(f"GemLite 1-bit src must be uint8 [K/8, N] = ({K // 8}, {N}), got {tuple(src.shape)}")
    words = torch.empty((N, words_per_row(K, 1)), dtype=torch.int32, device=src.device)
    st = lib().lowbit_import_binary_gemlite(ctypes.c_void_p(src.data_ptr()), ctypes.c_void_p(words.data_ptr()), N, K,
                                            ctypes.c_void_p(_stream_ptr(src.device)))
    _check(st, "lowbit_import_binary_gemlite")
    return words


def workspace_size(M: int, N: int, K: int, g: int = 64, bits: int = 2) -> int:
    """Bytes of workspace lowbit_gemm_ex can use for this shape (0: none needed)."""
    return int(lib().lowbit_workspace_size(M, N, K, g, bits))


def gemm(x, words, scales, g: int, bits: int, out=None, workspace=None):
    """Y[M, N] = X[M, K] . dequant(W)[N, K]^T in bf16 (see include/lowbit.h).

    `workspace`: an optional zero-filled device tensor (any dtype) of at least
    workspace_size(M, N, K, g, bits) bytes; it lets skinny problems split K across
    workgroups (lowbit_gemm_ex).  Reuse it between calls; do not share it between calls
    that run concurrently."""
    torch = _torch()
    _require(x, torch.bfloat16, "x")
    _require(words, torch.int32, "words")
    _require(scales, torch.float16, "scales")
    M, K = x.shape
    N = words.shape[0]
    if words.shape[1] != words_per_row(K, bits):
        raise ValueError(f"words must be [N, K*bits/32] = [{N}, {words_per_row(K, bits)}], got {tuple(words.shape)}")
    if K % g or tuple(scales.shape) != (N, K // g):
        raise ValueError(f"scales must be [N, K/g] = [{N}, {K // g if g else 0}], got {tuple(scales.shape)}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _require(out, torch.bfloat16, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N]")
    if workspace is None:
        st = lib().lowbit_gemm(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(words.data_ptr()),
                               ctypes.c_void_p(scales.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                               M, N, K, g, bits, ctypes.c_void_p(_stream_ptr(x.device)))
        _check(st, "lowbit_gemm")
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor")
        nbytes = workspace.numel() * workspace.element_size()
        st = lib().lowbit_gemm_ex(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(words.data_ptr()),
                                  ctypes.c_void_p(scales.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                  M, N, K, g, bits, ctypes.c_void_p(workspace.data_ptr()), nbytes,
                                  ctypes.c_void_p(_stream_ptr(x.device)))
        _check(st, "lowbit_gemm_ex")
    return out


NOALLOC_SCRATCH_BYTES = 4096 + 512 * 16 * 1024  # LOWBIT_NOALLOC_SCRATCH_BYTES of include/lowbit.h


def gemm_noalloc(x, words, scales, g: int, bits: int, out):
    """lowbit_gemm_noalloc: lowbit_gemm_ex on the library's static per-GPU scratch, for callers
    that cannot allocate (`out` is required: this call allocates nothing).  Calls on one GPU
    share the scratch and must not overlap."""
    torch = _torch()
    _require(x, torch.bfloat16, "x")
    _require(words, torch.int32, "words")
    _require(scales, torch.float16, "scales")
    _require(out, torch.bfloat16, "out")
    M, K = x.shape
    N = words.shape[0]
    if words.shape[1] != words_per_row(K, bits):
        raise ValueError(f"words must be [N, K*bits/32] = [{N}, {words_per_row(K, bits)}], got {tuple(words.shape)}")
    if K % g or tuple(scales.shape) != (N, K // g):
        raise ValueError(f"scales must be [N, K/g] = [{N}, {K // g if g else 0}], got {tuple(scales.shape)}")
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    st = lib().lowbit_gemm_noalloc(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(words.data_ptr()),
                                   ctypes.c_void_p(scales.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                   M, N, K, g, bits, ctypes.c_void_p(_stream_ptr(x.device)))
    _check(st, "lowbit_gemm_noalloc")
    return out


class Problem(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("S", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("g", ctypes.c_int32), ("bits", ctypes.c_int32)]


def gemm_swiglu(x, words, scales, g: int, bits: int, out=None):
    """Y[M, N] = silu(X . dequant(Wg)^T) * (X . dequant(Wu)^T) in bf16, with `words` / `scales`
    holding 2N rows: gate rows [0, N), then up rows [N, 2N) (lowbit_gemm_swiglu)."""
    torch = _torch()
    _require(x, torch.bfloat16, "x")
    _require(words, torch.int32, "words")
    _require(scales, torch.float16, "scales")
    M, K = x.shape
    N2 = words.shape[0]
    if N2 % 2:
        raise ValueError(f"words must hold 2N rows (gate then up), got {N2}")
    N = N2 // 2
    if words.shape[1] != words_per_row(K, bits):
        raise ValueError(f"words must be [2N, K*bits/32] = [{N2}, {words_per_row(K, bits)}], got {tuple(words.shape)}")
    if K % g or tuple(scales.shape) != (N2, K // g):
        raise ValueError(f"scales must be [2N, K/g] = [{N2}, {K // g if g else 0}], got {tuple(scales.shape)}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _require(out, torch.bfloat16, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N]")
    st = lib().lowbit_gemm_swiglu(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(words.data_ptr()),
                                  ctypes.c_void_p(scales.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                  M, N, K, g, bits, ctypes.c_void_p(_stream_ptr(x.device)))
    _check(st, "lowbit_gemm_swiglu")
    return out


def gemm_residual(x, words, scales, g: int, bits: int, residual, gate, out=None):
    """Y[M, N] = residual + gate[n] * (X . dequant(W)^T) in bf16 (lowbit_gemm_residual).
    `out` may be `residual` itself (in-place update of the residual stream)."""
    torch = _torch()
    _require(x, torch.bfloat16, "x")
    _require(words, torch.int32, "words")
    _require(scales, torch.float16, "scales")
    _require(residual, torch.bfloat16, "residual")
    _require(gate, torch.bfloat16, "gate", ndim=1)
    M, K = x.shape
    N = words.shape[0]
    if words.shape[1] != words_per_row(K, bits):
        raise ValueError(f"words must be [N, K*bits/32] = [{N}, {words_per_row(K, bits)}], got {tuple(words.shape)}")
    if K % g or tuple(scales.shape) != (N, K // g):
        raise ValueError(f"scales must be [N, K/g] = [{N}, {K // g if g else 0}], got {tuple(scales.shape)}")
    if tuple(residual.shape) != (M, N) or tuple(gate.shape) != (N,):
        raise ValueError("residual must be [M, N] and gate [N]")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _require(out, torch.bfloat16, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N]")
    st = lib().lowbit_gemm_residual(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(words.data_ptr()),
                                    ctypes.c_void_p(scales.data_ptr()), ctypes.c_void_p(residual.data_ptr()),
                                    ctypes.c_void_p(gate.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                    M, N, K, g, bits, ctypes.c_void_p(_stream_ptr(x.device)))
    _check(st, "lowbit_gemm_residual")
    return out


def _problem_array(problems):
    torch = _torch()
    if len(problems) > MAX_BATCH:
        raise ValueError(f"at most {MAX_BATCH} problems per call")
    arr = (Problem * max(1, len(problems)))()
    dev = None
    for i, (x, w, s, y, g, bits) in enumerate(problems):
        _require(x, torch.bfloat16, "x")
        _require(w, torch.int32, "words")
        _require(s, torch.float16, "scales")
        _require(y, torch.bfloat16, "out")
        M, K = x.shape
        N = w.shape[0]
        if w.shape[1] != words_per_row(K, bits) or tuple(s.shape) != (N, K // g) or tuple(y.shape) != (M, N):
            raise ValueError(f"problem {i}: inconsistent shapes")
        dev = x.device
        arr[i] = Problem(x.data_ptr(), w.data_ptr(), s.data_ptr(), y.data_ptr(), M, N, K, g, bits)
    return arr, dev


def batched_workspace_size(problems: Sequence[Tuple["object", "object", "object", "object", int, int]]) -> int:
    """Bytes of workspace gemm_batched(..., workspace=...) can use (0: none needed)."""
    arr, _ = _problem_array(problems)
    return int(lib().lowbit_batched_workspace_size(arr, len(problems))) if problems else 0


def gemm_batched(problems: Sequence[Tuple["object", "object", "object", "object", int, int]],
                 workspace=None) -> None:
    """Run independent GEMMs [(x, words, scales, out, g, bits), ...] as grouped launches.
    Outputs are written in place; all tensors on the same device.  `workspace`: as for gemm()
    (size from batched_workspace_size)."""
    arr, dev = _problem_array(problems)
    if not problems:
        return
    stream = ctypes.c_void_p(_stream_ptr(dev))
    if workspace is None:
        st = lib().lowbit_gemm_batched(arr, len(problems), stream)
        _check(st, "lowbit_gemm_batched")
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor")
        st = lib().lowbit_gemm_batched_ex(arr, len(problems), ctypes.c_void_p(workspace.data_ptr()),
                                          workspace.numel() * workspace.element_size(), stream)
        _check(st, "lowbit_gemm_batched_ex")


# ---- operators around the packed linears ----
# Their calls take a few microseconds on the device at small sizes, so the checks below look at the ordinary case first and
# the descriptors are packed bytes: a call costs the host about as much as a torch operation.

_get = None  # (torch.Tensor, current raw stream of a device index, current device index), once torch is there


def _env():
    global _get
    if _get is None:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
        torch.cuda.init()
        _get = (torch.Tensor, raw, getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device))
    return _get


def _heads(t, name: str, ndim: int) -> None:
    """A bf16 device tensor [..., heads, head_dim] whose last dimension is contiguous (any other strides)."""
    torch = _torch()
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.dim() == ndim and t.is_cuda and (
            t.stride(-1) == 1 or t.shape[-1] == 1):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    raise ValueError(f"{name} must be contiguous along its last dimension")


def _plain(t, dtype, name: str, ndim: int, like) -> int:
    """The address of a contiguous tensor of that type on the device of `like`."""
    if not (t.__class__ is like.__class__ and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()
            and t.get_device() == like.get_device() and t.is_cuda):
        _require(t, dtype, name, ndim)
        _same_device(like, ((name, t),))
    return t.data_ptr()


def _same_device(first, named) -> None:
    """Every tensor of `named` on the device of `first` (the kernel runs there)."""
    dev = first.get_device()
    for name, t in named:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} must be on {first.device}, got {t.device}")


def _call(function: str, like, *args) -> None:
    """Calls the library with the current stream of the tensors' device, that device being current (a launch goes
    to the current device)."""
    _, raw_stream, current = _env()
    dev = like.get_device()
    if dev == current():
        st = getattr(lib(), function)(*args, raw_stream(dev))
    else:
        with _torch().cuda.device(dev):
            st = getattr(lib(), function)(*args, raw_stream(dev))
    if st:
        _check(st, function)


def _strides(t):
    """Strides of every dimension but the last, 0 for dimensions of one element (whose stride says nothing)."""
    n, s = t.shape, t.stride()
    if len(n) == 3:
        return (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0)
    return (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)


def _workspace(workspace, like):
    """(address, bytes) of an optional workspace."""
    if workspace is None:
        return 0, 0
    if not isinstance(workspace, _TORCH.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor")
        _same_device(like, (("workspace", workspace),))
    return workspace.data_ptr(), workspace.nbytes


def _output(out, shape, like):
    """`out`, checked, or a new bf16 tensor of that shape."""
    torch = _torch()
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=like.device)
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a torch.Tensor")
    if out.shape != shape:
        raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    return out


def lora_workspace_size(M: int, rank: int, N: Optional[int] = None, K: Optional[int] = None, g: int = 64, bits: int = 2) -> int:
    """Bytes of workspace that gemm_lora needs for M rows (0 for invalid arguments); with N and K, the bytes with which it
    can also split K across workgroups (lowbit_lora_split_workspace_size)."""
    if N is None or K is None:
        return int(lib().lowbit_lora_workspace_size(M, rank))
    return int(lib().lowbit_lora_split_workspace_size(M, N, K, g, bits, rank))


def gemm_lora(x, words, scales, g: int, bits: int, lora_a, lora_b, alpha, rows, out=None, workspace=None):
    """Y[m] = X[m] . dequant(W)^T + alpha[e] * (X[m] . A[e]^T) . B[e]^T with e = rows[m], in bf16
    (lowbit_gemm_lora): low-rank adapters of many requests beside one packed weight.  lora_a bf16 [adapters, rank, K],
    lora_b bf16 [adapters, N, rank], alpha fp32 [adapters], rows int32 [M] (-1: no adapter).

    `workspace`: a device tensor of at least lora_workspace_size(M, rank) bytes, zero-filled before its first use (reuse
    it between calls; do not share it between calls that run concurrently); that much is allocated for the call if None.
    With the bytes that lora_workspace_size says for N and K too, K can be split (509 x 3072 x 9216 binary: 55 us, 68 without)."""
    torch = _torch()
    bf16 = torch.bfloat16
    _require(x, bf16, "x")
    M, K = x.shape
    px = x.data_ptr()
    pw = _plain(words, torch.int32, "words", 2, x)
    ps = _plain(scales, torch.float16, "scales", 2, x)
    pa = _plain(lora_a, bf16, "lora_a", 3, x)
    pb = _plain(lora_b, bf16, "lora_b", 3, x)
    pl = _plain(alpha, torch.float32, "alpha", 1, x)
    pr = _plain(rows, torch.int32, "rows", 1, x)
    N, per_row = words.shape
    E, rank, ka = lora_a.shape
    if per_row != words_per_row(K, bits):
        raise ValueError(f"words must be [N, K*bits/32] = [{N}, {words_per_row(K, bits)}], got {tuple(words.shape)}")
    if K % g or scales.shape != (N, K // g):
        raise ValueError(f"scales must be [N, K/g] = [{N}, {K // g if g else 0}], got {tuple(scales.shape)}")
    if ka != K or lora_b.shape != (E, N, rank):
        raise ValueError(f"lora_a must be [adapters, rank, {K}] and lora_b [adapters, {N}, rank], got "
                         f"{tuple(lora_a.shape)} and {tuple(lora_b.shape)}")
    if alpha.shape[0] != E or rows.shape[0] != M:
        raise ValueError(f"alpha must be [{E}] and rows [{M}]")
    out = _output(out, (M, N), x)
    po = _plain(out, bf16, "out", 2, x)
    if workspace is None:
        workspace = torch.zeros(lora_workspace_size(M, rank), dtype=torch.uint8, device=x.device)
    ws, nbytes = _workspace(workspace, x)
    _call("lowbit_gemm_lora", x, px, pw, ps, po, M, N, K, g, bits, pa, pb, pl, pr, E, rank, ws, nbytes)
    return out


_QK_PROBLEM = struct.Struct("@8P9q9if0q")  # lowbit_qk_problem of include/lowbit.h


def rope_freqs(axis_dims: Sequence[int], theta: float = 10000.0, device="cuda"):
    """fp32 [sum(axis_dims) / 2]: theta^(-2i / axis_dims[a]) for pair i of each axis a, the usual choice of
    qk_norm_rope's `freqs` (any other, e.g. scaled for longer contexts, can be passed as well)."""
    torch = _torch()
    parts = [theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in axis_dims]
    return (torch.cat(parts) if parts else torch.empty(0, dtype=torch.float64)).to(torch.float32).to(device)


def qk_norm_rope(q, k, positions, freqs, axis_dims: Sequence[int], q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = True, q_out=None, k_out=None):
    """RMS norm of every head of q [tokens, q_heads, D] and k [tokens, k_heads, D] (bf16, any strides of
    whole 16-byte pieces, e.g. views of a fused QKV output) and their rotation by `positions` (int32 [tokens, axes]) and `freqs`
    (fp32, radians per unit position and pair), in one pass (lowbit_qk_norm_rope).

    A weight of None leaves that tensor unnormed; axis_dims = () leaves both unturned (positions and
    freqs may then be None).  `interleaved` pairs neighbouring elements, otherwise element i goes with i +
    sum(axis_dims) / 2.  q_out / k_out may be q / k themselves.  Returns (q_out, k_out)."""
    torch = _torch()
    _heads(q, "q", 3)
    _heads(k, "k", 3)
    T, Hq, D = q.shape
    Tk, Hk, Dk = k.shape
    if Tk != T or Dk != D:
        raise ValueError(f"k must be [{T}, heads, {D}], got {tuple(k.shape)}")
    axes = len(axis_dims)
    if axes > 4:
        raise ValueError("at most 4 axes")
    pp = pf = 0
    if axes:
        pp = _plain(positions, torch.int32, "positions", 2, q)
        pf = _plain(freqs, torch.float32, "freqs", 1, q)
        if positions.shape != (T, axes):
            raise ValueError(f"positions must be [{T}, {axes}], got {tuple(positions.shape)}")
        if 2 * freqs.shape[0] != sum(axis_dims):
            raise ValueError(f"freqs must hold sum(axis_dims) / 2 = {sum(axis_dims) // 2} values, got {freqs.shape[0]}")
    pwq = pwk = 0
    if q_weight is not None:
        pwq = _plain(q_weight, torch.bfloat16, "q_weight", 1, q)
        if q_weight.shape[0] != D:
            raise ValueError(f"q_weight must be [{D}]")
    if k_weight is not None:
        pwk = _plain(k_weight, torch.bfloat16, "k_weight", 1, q)
        if k_weight.shape[0] != D:
            raise ValueError(f"k_weight must be [{D}]")
    q_out, k_out = _output(q_out, q.shape, q), _output(k_out, k.shape, q)
    _heads(q_out, "q_out", 3)
    _heads(k_out, "k_out", 3)
    _same_device(q, (("k", k), ("q_out", q_out), ("k_out", k_out)))
    dims = (*axis_dims, 0, 0, 0, 0)
    p = _QK_PROBLEM.pack(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), pwq, pwk, pp, pf, T,
                         *_strides(q), *_strides(k), *_strides(q_out), *_strides(k_out), Hq, Hk, D, axes,
                         dims[0], dims[1], dims[2], dims[3], 1 if interleaved else 0, eps)
    _call("lowbit_qk_norm_rope", q, p)
    return q_out, k_out


_ATTENTION_PROBLEM = struct.Struct("@7P16q4if0q")  # lowbit_attention_problem of include/lowbit.h


def _attention_problem(q, k, v, key_mask, key_lens, causal, q_start, scale, out):
    torch = _torch()
    _heads(q, "q", 4)
    _heads(k, "k", 4)
    _heads(v, "v", 4)
    B, Lq, Hq, D = q.shape
    _, Lk, Hk, _ = k.shape
    if k.shape != (B, Lk, Hk, D) or v.shape != k.shape:
        raise ValueError(f"k and v must be [{B}, keys, kv_heads, {D}], got {tuple(k.shape)} and {tuple(v.shape)}")
    pm = pn = pq = mask_batch = 0
    if key_mask is not None:
        if not isinstance(key_mask, torch.Tensor) or key_mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("key_mask must be a bool or uint8 torch.Tensor")
        if key_mask.shape != (B, Lk) or (Lk > 1 and key_mask.stride(1) != 1):
            raise ValueError(f"key_mask must be [{B}, {Lk}], contiguous along the keys")
        if not key_mask.is_cuda:
            raise ValueError("key_mask must be on a GPU")
        pm, mask_batch = key_mask.data_ptr(), key_mask.stride(0) if B > 1 else 0
    if key_lens is not None:
        pn = _plain(key_lens, torch.int32, "key_lens", 1, q)
        if key_lens.shape[0] != B:
            raise ValueError(f"key_lens must be [{B}]")
    if q_start is not None and causal:  # positions matter to the causal rule only
        pq = _plain(q_start, torch.int32, "q_start", 1, q)
        if q_start.shape[0] != B:
            raise ValueError(f"q_start must be [{B}]")
    po, so = 0, (Lq * Hq * D, Hq * D, D)
    if out is not None:
        _heads(out, "out", 4)
        po, so = out.data_ptr(), _strides(out)
    _same_device(q, (("k", k), ("v", v), ("key_mask", key_mask), ("out", out)))
    return _ATTENTION_PROBLEM.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), po, pm, pn, pq, B, Lq, Lk, *_strides(q),
                                   *_strides(k), *_strides(v), *so, mask_batch, Hq, Hk, D, 1 if causal else 0,
                                   scale if scale is not None else D ** -0.5 if D else 1.0)


def attention_workspace_size(q, k, v) -> int:
    """Bytes of workspace attention(q, k, v, ...) can use (0: none)."""
    return int(lib().lowbit_attention_workspace_size(_attention_problem(q, k, v, None, None, False, None, None, None)))


def attention(q, k, v, key_mask=None, key_lens=None, causal: bool = False, q_start=None, scale=None, out=None,
              workspace=None):
    """softmax(scale * q k^T) v in bf16 (lowbit_attention): q [batch, q_len, q_heads, D], k and v [batch, kv_len,
    kv_heads, D] with any strides of whole 16-byte pieces (views of a fused QKV output, a cache), D 64 or 128, q_heads a multiple of
    kv_heads.  Query t takes key j where key_mask[b, j] (bool), j < key_lens[b] and, if causal, j <= q_start[b] + t (None: 0);
    a query without keys gets zeros.  scale: 1 / sqrt(D) by default.

    `workspace`: an optional device tensor of at least attention_workspace_size(q, k, v) bytes, zero-filled before its
    first use, with which few rows over many keys run split along the keys: pass one when decoding (one token over 40007 keys, 8 kv
    heads of 128: 36 us, 411 without).  Reuse it between calls; do not share it between calls that run concurrently."""
    if out is None:
        _heads(q, "q", 4)
    out = _output(out, q.shape, q)
    p = _attention_problem(q, k, v, key_mask, key_lens, causal, q_start, scale, out)
    ws, nbytes = _workspace(workspace, q)
    _call("lowbit_attention", q, p, ws, nbytes)
    return out


# ---- decoding: a paged cache, attention over it, matrix-vector products ----

CACHE_ATTENTION_WORKSPACE_BYTES = 17043456  # LOWBIT_CACHE_ATTENTION_WORKSPACE_BYTES: enough for every call
_CACHE = struct.Struct("@4Pq4i0q")  # lowbit_cache of include/lowbit.h
_CACHE_ATTENTION_PROBLEM = struct.Struct("@4Pq4i6P10qif0q")  # lowbit_cache_attention_problem


class KVCache:
    """Keys and values of many requests in pages (lowbit_cache): k and v [pages, kv_heads, page_size, row], uint8 with head_dim * bits / 8
    bytes a row at 8 and 4 bits, bf16 with head_dim elements at 16; k_scales and v_scales bf16, [pages, kv_heads, page_size] at 8 bits,
    [pages, kv_heads, page_size, head_dim / 64, 2] at 4, None at 16.  page_size 16 .. 256 (a power of two), head_dim 64 or 128.
    kv_cache() allocates one.  The order inside a page's head is the library's: cache_write and cache_read convert."""

    __slots__ = ("k", "v", "k_scales", "v_scales", "bits", "shape")

    def __init__(self, k, v, k_scales=None, v_scales=None, bits: int = 8):
        torch = _torch()
        if bits not in (4, 8, 16):
            raise ValueError(f"bits must be 4, 8 or 16, got {bits}")
        dtype = torch.bfloat16 if bits == 16 else torch.uint8
        _require(k, dtype, "k", 4)
        shape = k.shape
        pages, heads, page, row = shape
        dev = k.get_device()
        if not (_fits(v, dtype, dev) and v.shape == shape):
            _plain(v, dtype, "v", 4, k)
            raise ValueError(f"v must be {tuple(shape)}, got {tuple(v.shape)}")
        dim = row if bits == 16 else row * 8 // bits
        if bits == 16:
            if k_scales is not None or v_scales is not None:
                raise ValueError("a 16-bit cache has no scales")
        else:
            want = (pages, heads, page) if bits == 8 else (pages, heads, page, dim // 64, 2)
            bf16 = torch.bfloat16
            if not (_fits(k_scales, bf16, dev) and _fits(v_scales, bf16, dev) and k_scales.shape == want and v_scales.shape == want):
                for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
                    _plain(t, bf16, name, len(want), k)
                    if t.shape != want:
                        raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}")
        self.k, self.v, self.k_scales, self.v_scales, self.bits = k, v, k_scales, v_scales, bits
        self.shape = (pages, heads, page, dim)

    def _fields(self):
        pages, heads, page, dim = self.shape
        if self.bits == 16:
            return self.k.data_ptr(), self.v.data_ptr(), 0, 0, pages, page, heads, dim, 16
        return (self.k.data_ptr(), self.v.data_ptr(), self.k_scales.data_ptr(), self.v_scales.data_ptr(), pages, page, heads, dim, self.bits)


def _fits(t, dtype, dev: int) -> bool:
    """Whether t is a contiguous tensor of that type on that device."""
    return isinstance(t, _TORCH.Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def kv_cache(pages: int, kv_heads: int, head_dim: int, bits: int = 8, page_size: int = 64, device="cuda") -> KVCache:
    """A new cache of zeros."""
    torch = _torch()
    if bits not in (4, 8, 16):
        raise ValueError(f"bits must be 4, 8 or 16, got {bits}")
    if head_dim not in (64, 128):
        raise ValueError(f"head_dim must be 64 or 128, got {head_dim}")
    row = (pages, kv_heads, page_size, head_dim if bits == 16 else head_dim * bits // 8)
    k, v = (torch.zeros(row, dtype=torch.bfloat16 if bits == 16 else torch.uint8, device=device) for _ in range(2))
    if bits == 16:
        return KVCache(k, v, bits=16)
    scales = row[:3] if bits == 8 else (*row[:3], head_dim // 64, 2)
    return KVCache(k, v, *(torch.zeros(scales, dtype=torch.bfloat16, device=device) for _ in range(2)), bits=bits)


def _row_strides(t, name: str, shape, dev: int):
    """(token, head) strides of bf16 rows `shape` = [tokens, heads, D] whose elements lie together, 0 for dimensions of one."""
    if t.dtype is not _torch().bfloat16 or t.get_device() != dev or t.shape != shape:
        _heads(t, name, 3)
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be on the cache's device, got {t.device}")
    token, head, one = t.stride()
    if one != 1:
        _heads(t, name, 3)
    return token if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def _require_cache(cache) -> None:
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")


def _cache_rows(function: str, cache: KVCache, k, v, slots) -> None:
    _require_cache(cache)
    like = cache.k
    dev = like.get_device()
    at = _plain(slots, _torch().int32, "slots", 1, like)
    _, heads, _, dim = cache.shape
    shape = (slots.shape[0], heads, dim)
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, _TORCH.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    ks, vs = _row_strides(k, "k", shape, dev), _row_strides(v, "v", shape, dev)
    _call(function, like, _CACHE.pack(*cache._fields()), k.data_ptr(), v.data_ptr(), shape[0], *ks, *vs, at)


def cache_write(cache: KVCache, k, v, slots) -> None:
    """Quantises k and v [tokens, kv_heads, head_dim] (bf16, any strides of whole 16-byte pieces, e.g. views of a fused QKV output) into the
    cache's slots (int32 [tokens]: page * page_size + place; -1 leaves a row out; those of one call differ) (lowbit_cache_write)."""
    _cache_rows("lowbit_cache_write", cache, k, v, slots)


def cache_read(cache: KVCache, slots, k_out=None, v_out=None):
    """The rows at `slots` (int32 [tokens]) as bf16 [tokens, kv_heads, head_dim] (lowbit_cache_read): (k_out, v_out).  Rows whose slot
    is outside the cache are left as they were (zeros where the output is made here).  At 8 and 4 bits a row read back and written again is
    quantised a second time."""
    if k_out is None or v_out is None:
        torch = _torch()
        _require_cache(cache)
        _plain(slots, torch.int32, "slots", 1, cache.k)
        shape = (slots.shape[0], cache.shape[1], cache.shape[3])
        k_out, v_out = (torch.zeros(shape, dtype=torch.bfloat16, device=cache.k.device) if t is None else t for t in (k_out, v_out))
    _cache_rows("lowbit_cache_read", cache, k_out, v_out, slots)
    return k_out, v_out


def _cache_attention_problem(q, cache, page_table, key_lens, q_lens, tree, kv_len, scale, out):
    torch = _torch()
    int32 = torch.int32
    _heads(q, "q", 4)
    _require_cache(cache)
    B, Lq, Hq, D = shape = q.shape
    _, _, page, dim = cache.shape
    dev = q.get_device()
    if D != dim:
        raise ValueError(f"q must be [batch, q_len, q_heads, {dim}], got {tuple(shape)}")
    if cache.k.get_device() != dev:
        raise ValueError(f"cache must be on {q.device}, got {cache.k.device}")
    pt = pk = pq = ptree = po = of_row = 0
    if page_table is not None:
        if not (isinstance(page_table, torch.Tensor) and page_table.dtype is int32 and page_table.dim() == 2 and page_table.get_device() == dev):
            _plain(page_table, int32, "page_table", 2, q)
        pt = page_table.data_ptr()
        pk = key_lens.data_ptr() if _fits(key_lens, int32, dev) and key_lens.dim() == 1 else _plain(key_lens, int32, "key_lens", 1, q)
        rows, pages = page_table.shape
        of_row, of_page = page_table.stride()
        if of_page != 1 and pages > 1:
            raise ValueError("page_table must be contiguous along the pages")
        if rows != B or key_lens.shape[0] != B:
            raise ValueError(f"page_table must be [{B}, pages] and key_lens [{B}]")
        if kv_len is None:
            kv_len = pages * page
        elif kv_len > pages * page:
            raise ValueError(f"page_table holds {pages * page} keys of a request, fewer than kv_len = {kv_len}")
    if q_lens is not None:
        pq = _plain(q_lens, int32, "q_lens", 1, q)
        if q_lens.shape[0] != B:
            raise ValueError(f"q_lens must be [{B}]")
    if tree is not None:
        ptree = _plain(tree, torch.int64, "tree", 2, q)
        if tree.shape != (B, Lq):
            raise ValueError(f"tree must be [{B}, {Lq}]")
    qb, qt, qh, _ = q.stride()
    ob, ot, oh = Lq * Hq * D, Hq * D, D
    if out is not None:
        if out.dtype is not torch.bfloat16 or out.get_device() != dev or out.stride(3) != 1:
            _heads(out, "out", 4)
            _same_device(q, (("out", out),))
        po = out.data_ptr()
        ob, ot, oh, _ = out.stride()
    if B <= 1:  # strides along dimensions of one say nothing
        qb = ob = 0
    if Lq <= 1:
        qt = ot = 0
    if Hq <= 1:
        qh = oh = 0
    return _CACHE_ATTENTION_PROBLEM.pack(*cache._fields(), q.data_ptr(), po, pt, pk, pq, ptree, B, Lq, kv_len, qb, qt, qh, ob, ot, oh, of_row if B > 1 else 0, Hq,
                                         scale if scale is not None else D ** -0.5)


def cache_attention_workspace_size(q, cache: KVCache, kv_len: int) -> int:
    """Bytes of workspace that cache_attention can use for q and this many keys at most (0: none).  Fewer requests can use more (their keys
    are split further): CACHE_ATTENTION_WORKSPACE_BYTES cover every call."""
    return int(lib().lowbit_cache_attention_workspace_size(_cache_attention_problem(q, cache, None, None, None, None, kv_len, None, None)))


def cache_attention(q, cache: KVCache, page_table, key_lens, q_lens=None, tree=None, kv_len: Optional[int] = None, scale=None, out=None,
                    workspace=None):
    """Attention of each request's last tokens over its keys and values in the cache, in bf16 (lowbit_cache_attention): q [batch, q_len,
    q_heads, head_dim] (any strides of whole 16-byte pieces), page_table int32 [batch, pages of a request] (rows at any stride, e.g. part of a wider
    table), key_lens int32 [batch]: keys, the new tokens' among them (cache_write puts them there first).  Every new token takes the keys before
    the new ones and, of those, the ones up to itself, or where bit i of tree[b, t] (int64 [batch, q_len], q_len <= 64) is set: a tree of drafted
    tokens, each with its ancestors and itself.  q_lens int32 [batch]: requests with fewer new tokens than q_len; rows of `out` past them are left
    as they were (zeros where the output is made here).  kv_len: the most keys a request has in this call, if that is less than the table holds (it
    chooses how the keys are split; a longer key_lens counts as kv_len).  scale: 1 / sqrt(head_dim) by default.

    `workspace`: an optional device tensor of at least cache_attention_workspace_size(q, cache, kv_len) bytes, zero-filled before its first use, with
    which few rows over many keys run split along the keys: pass one when decoding (one of CACHE_ATTENTION_WORKSPACE_BYTES where batches change).
    Reuse it between calls; do not share it between calls that run concurrently."""
    if page_table is None or key_lens is None:
        raise TypeError("page_table and key_lens must be int32 tensors")
    if out is None:
        _heads(q, "q", 4)
        torch = _torch()
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) if q_lens is None else torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
    elif out.__class__ is not q.__class__ or out.shape != q.shape:
        _heads(q, "q", 4)
        out = _output(out, q.shape, q)
    p = _cache_attention_problem(q, cache, page_table, key_lens, q_lens, tree, kv_len, scale, out)
    ws, nbytes = _workspace(workspace, q)
    _call("lowbit_cache_attention", q, p, ws, nbytes)
    return out


def gemv_affine(x, words, scales, biases, g: int, residual=None, swiglu: bool = False, out=None):
    """gemm_affine for up to 16 rows (lowbit_gemv_affine): Y = X . W^T (+ residual), W = S * u + B with `words` from pack_u4.  swiglu: words,
    scales and biases hold 2N rows, gate then up, and Y = silu(X . Wg^T) * (X . Wu^T) (+ residual).  residual bf16 [M, N], may be `out`.  An
    infinite element of x leaves its row of Y without a finite number."""
    torch = _torch()
    _require(x, torch.bfloat16, "x")
    M, K = x.shape
    pw = _plain(words, torch.int32, "words", 2, x)
    ps = _plain(scales, torch.float16, "scales", 2, x)
    pb = _plain(biases, torch.float16, "biases", 2, x)
    rows, per_row = words.shape
    if g not in (64, 128):
        raise ValueError(f"g must be 64 or 128, got {g}")
    if per_row != K // 8 or K % g or scales.shape != (rows, K // g) or biases.shape != scales.shape:
        raise ValueError(f"words must be [{rows}, K/8], scales and biases [{rows}, K/g] with K = {K}, got {tuple(words.shape)}, "
                         f"{tuple(scales.shape)} and {tuple(biases.shape)}")
    if swiglu and rows % 2:
        raise ValueError(f"words must hold 2N rows (gate then up), got {rows}")
    N = rows // 2 if swiglu else rows
    pr = 0
    if residual is not None:
        pr = _plain(residual, torch.bfloat16, "residual", 2, x)
        if residual.shape != (M, N):
            raise ValueError(f"residual must be [{M}, {N}]")
    out = _output(out, (M, N), x)
    po = _plain(out, torch.bfloat16, "out", 2, x)
    _call("lowbit_gemv_affine", x, x.data_ptr(), pw, ps, pb, pr, po, M, N, K, g, 1 if swiglu else 0)
    return out


def check_gemm_args(x_ptr: int, w_ptr: int, s_ptr: int, y_ptr: int, M: int, N: int, K: int, g: int,
                    bits: int) -> int:
    """Host-only validation (no HIP call); returns the status code lowbit_gemm would return."""
    return lib().lowbit_check_gemm_args(ctypes.c_void_p(x_ptr), ctypes.c_void_p(w_ptr), ctypes.c_void_p(s_ptr),
                                        ctypes.c_void_p(y_ptr), M, N, K, g, bits)


def variant(M: int, N: int, K: int, g: int = 64, bits: int = 2) -> str:
    """Name of the kernel variant lowbit_gemm picks for this shape."""
    return lib().lowbit_gemm_variant(M, N, K, g, bits).decode()


def status_string(status: int) -> str:
    return lib().lowbit_status_string(status).decode()


def version() -> int:
    return lib().lowbit_version()
