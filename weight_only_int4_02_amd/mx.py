"""Microscaled 4-bit floating point (MXFP4): quantization, products, products
grouped by expert.

    X [.., K] fp16, bf16 or fp32       -> quantize()     -> MXTensor
    codes, scales of a checkpoint      -> tensor()       -> MXTensor
    MXTensor                           -> dequantize()   -> X [.., K]
    MXTensor [N, K] or [E, N, K]       -> weight()       -> MXWeight (device layout)
    X [M, K] or MXTensor, MXWeight     -> gemm()         -> Y [M, N]
    X, MXWeight of E, offsets          -> grouped_gemm() -> Y [R, N]

The format is that of the Open Compute Project's microscaling specification:
blocks of 32 columns, 4-bit elements (sign; 0, 0.5, 1, 1.5, 2, 3, 4 or 6), a
power of two a block.  A thin binding over libw4a16.so (C ABI in
include/w4a16_mx.h): arguments are checked and marshalled here, every step runs
in the library's HIP kernels on the current stream.  Serving only: no
gradients are formed.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass
from typing import Optional

import torch

from . import _raise, lib
from .moe import check, stream_of

BLOCK = 32

# Symbols of include/w4a16_mx.h.
EXPORTS = ("w4a16_mx_quantize", "w4a16_mx_check_quantize_args", "w4a16_mx_dequantize",
           "w4a16_mx_check_dequantize_args", "w4a16_mx_weight_size", "w4a16_mx_weight",
           "w4a16_mx_check_weight_args", "w4a16_mx_gemm_workspace_size", "w4a16_mx_gemm",
           "w4a16_mx_check_gemm_args",
           "w4a16_mx_grouped_gemm", "w4a16_mx_check_grouped_gemm_args", "w4a16_mx_kernel")

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_DTYPES16 = {torch.float16: 0, torch.bfloat16: 1}

_bound = None


def _mx():
    """libw4a16.so with this module's argument types set."""
    global _bound
    if _bound is None:
        L = lib()
        P, I64, I32, PSZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)
        args = {"quantize": [P, I32, I64, I64, P, P], "dequantize": [P, P, I64, I64, I32, P],
                "weight": [P, P, I64, I64, I64, P, P],
                "gemm": [P, P, I32, I64, I64, P, P, I64, I32, P, P, ctypes.c_size_t],
                "grouped_gemm": [P, P, I32, I64, I64, P, I64, P, I64, P, P, I64, I32, P]}
        for name, types in args.items():
            getattr(L, f"w4a16_mx_{name}").argtypes = types + [P]
            getattr(L, f"w4a16_mx_check_{name}_args").argtypes = types
        L.w4a16_mx_gemm_workspace_size.argtypes = [I64, I64, I64, I32, PSZ]
        L.w4a16_mx_kernel.argtypes = [I64, I64, I64, I64, I32, I32, ctypes.POINTER(I32)]
        L.w4a16_mx_weight_size.argtypes = [I64, I64, I64, PSZ, PSZ]
        for name in EXPORTS:
            getattr(L, name).restype = I32
        _bound = L
    return _bound


@dataclass
class MXTensor:
    """MXFP4 rows, owned by torch tensors: codes uint8 [4 KG, .., 64] (of 128
    columns the 64 bytes of each row, two columns a byte, the first in the low half)
    and scales uint8 [KG, .., 16] (of 512 columns the 16 scales of each row:
    2^(b - 127), 255 for NaN), KG = ceil(K / 512); columns from K on hold zeros.
    dtype: the type dequantize() gives where none is named, and products too (bf16
    for fp32)."""
    codes: torch.Tensor
    scales: torch.Tensor
    K: int
    dtype: torch.dtype = torch.bfloat16

    @property
    def shape(self):
        return (*self.codes.shape[1:-1], self.K)


@dataclass
class MXWeight:
    """E matrices [N, K] in the device layout, owned by torch tensors."""
    q: torch.Tensor
    s: torch.Tensor
    E: int
    N: int
    K: int


def _float_type(dtype, types, name: str) -> int:
    if dtype not in types:
        raise TypeError(f"{name} must be one of {', '.join(str(t) for t in types)}, got {dtype}")
    return types[dtype]


def _type_of(x, types, name: str) -> int:
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return _float_type(x.dtype, types, name)


def _device_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be on a device")
    return device


def _check_tensor(t: MXTensor, name: str, device: int, rank: int) -> None:
    """The tensors of an MXTensor of `rank` dimensions hold what its shape needs
    (the kernels read them through bare pointers)."""
    codes, scales, KG = t.codes, t.scales, -(-t.K // 512)
    check(codes, name, torch.uint8, rank + 1, device)
    check(scales, name, torch.uint8, rank + 1, device)
    c, s = codes.shape, scales.shape
    if rank < 1 or KG < 1 or c[0] != 4 * KG or s[0] != KG or c[-1] != 64 or s[-1] != 16 or c[1:-1] != s[1:-1]:
        raise ValueError(f"{name}: codes must be [{4 * KG}, .., 64] and scales [{KG}, .., 16] for K = {t.K}, "
                         f"got {tuple(c)} and {tuple(s)}")


def quantize(x: torch.Tensor) -> MXTensor:
    """x [.., K] (fp16, bf16 or fp32, contiguous, K a multiple of 8) -> MXTensor.

    A block's scale is 2^(floor(log2 a) - 2) for its largest magnitude a; its
    elements are rounded to nearest, ties to even, beyond 6 scales to 6.  A block
    that holds an infinity or a NaN becomes NaN throughout.  There may be no
    rows; the last block of a row may be partial."""
    dt = _type_of(x, _DTYPES, "x")
    device = _device_of(x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    *rows, K = x.shape or (0,)
    if K < 1 or K % 8:
        raise ValueError("K must be a positive multiple of 8")
    stream = stream_of(device)
    KG = -(-K // 512)
    codes = torch.empty((4 * KG, *rows, 64), dtype=torch.uint8, device=x.device)
    scales = codes.new_empty((KG, *rows, 16))
    M = x.numel() // K
    if M:
        _raise(_mx().w4a16_mx_quantize(x.data_ptr(), dt, M, K, codes.data_ptr(), scales.data_ptr(), stream),
               "w4a16_mx_quantize")
    return MXTensor(codes, scales, K, x.dtype)


def dequantize(t: MXTensor, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The values of t [.., K], in dtype (t.dtype if None), each rounded once:
    exact in bf16 and fp32, but for magnitudes past the type's largest."""
    if not isinstance(t, MXTensor):
        raise TypeError("t must be an MXTensor")
    device = _device_of(t.codes, "t.codes")
    dtype = t.dtype if dtype is None else dtype
    dt = _float_type(dtype, _DTYPES, "dtype")
    _check_tensor(t, "t", device, t.codes.dim() - 1)
    stream = stream_of(device)
    out = torch.empty(t.shape, dtype=dtype, device=t.codes.device)
    M = out.numel() // t.K
    if M:
        _raise(_mx().w4a16_mx_dequantize(t.codes.data_ptr(), t.scales.data_ptr(), M, t.K, dt, out.data_ptr(),
                                         stream), "w4a16_mx_dequantize")
    return out


def tensor(codes: torch.Tensor, scales: torch.Tensor, K: Optional[int] = None,
           dtype: torch.dtype = torch.bfloat16) -> MXTensor:
    """codes uint8 [.., K/2] and scales uint8 [.., ceil(K/32)], as checkpoints hold
    them, on the device -> MXTensor (a copy, padded to whole slabs of 512 columns).
    K: twice the codes' last dimension if None."""
    device = _device_of(codes, "codes")
    if codes.dim() < 1:
        raise ValueError("codes must have at least one dimension")
    check(codes, "codes", torch.uint8, codes.dim(), device)
    check(scales, "scales", torch.uint8, codes.dim(), device)
    _float_type(dtype, _DTYPES, "dtype")
    K = 2 * codes.shape[-1] if K is None else K
    if K < 1 or K % 8:
        raise ValueError("K must be a positive multiple of 8")
    if (codes.shape[:-1] != scales.shape[:-1] or codes.shape[-1] != K // 2
            or scales.shape[-1] != -(-K // BLOCK)):
        raise ValueError("codes must be [.., K/2] and scales [.., ceil(K/32)]")
    KG = -(-K // 512)
    if codes.shape[-1] != 256 * KG:
        codes = torch.nn.functional.pad(codes, (0, 256 * KG - codes.shape[-1]))
    if scales.shape[-1] != 16 * KG:
        scales = torch.nn.functional.pad(scales, (0, 16 * KG - scales.shape[-1]), value=127)
    # (a copy in any case: where no padding is needed and the order is the same, a
    # view would change with the caller's buffers)
    codes = codes.unflatten(-1, (4 * KG, 64)).movedim(-2, 0).clone(memory_format=torch.contiguous_format)
    scales = scales.unflatten(-1, (KG, 16)).movedim(-2, 0).clone(memory_format=torch.contiguous_format)
    return MXTensor(codes, scales, K, dtype)


def weight_size(E: int, N: int, K: int):
    q, s = ctypes.c_size_t(), ctypes.c_size_t()
    _raise(_mx().w4a16_mx_weight_size(E, N, K, ctypes.byref(q), ctypes.byref(s)), "w4a16_mx_weight_size")
    return q.value, s.value


def weight(t: MXTensor) -> MXWeight:
    """An MXTensor [N, K], or [E, N, K] for E experts, in the products' layout."""
    if not isinstance(t, MXTensor):
        raise TypeError("t must be an MXTensor")
    device = _device_of(t.codes, "t.codes")
    if t.codes.dim() not in (3, 4):
        raise ValueError("t must be [N, K] or [E, N, K]")
    _check_tensor(t, "t", device, t.codes.dim() - 1)
    stream = stream_of(device)
    E, N = (1, *t.shape[:-1]) if t.codes.dim() == 3 else t.shape[:-1]
    qb, sb = weight_size(E, N, t.K)
    codes, scales = (x if x.data_ptr() % 16 == 0 else x.clone() for x in (t.codes, t.scales))
    q = torch.empty(qb, dtype=torch.uint8, device=codes.device)
    s = torch.empty(sb, dtype=torch.uint8, device=codes.device)
    _raise(_mx().w4a16_mx_weight(codes.data_ptr(), scales.data_ptr(), E, N, t.K, q.data_ptr(), s.data_ptr(),
                                 stream), "w4a16_mx_weight")
    return MXWeight(q, s, E, N, t.K)


def _check_weight(w: MXWeight, device: int) -> None:
    if not isinstance(w, MXWeight):
        raise TypeError("w must be an MXWeight")
    check(w.q, "w.q", torch.uint8, 1, device)
    check(w.s, "w.s", torch.uint8, 1, device)
    nt = w.E * -(-w.N // 16)
    if w.q.numel() < nt * -(-w.K // 128) * 1024 or w.s.numel() < nt * -(-w.K // 512) * 256:
        raise ValueError("MXWeight tensors are smaller than its shape needs")


def _activations(x, K: int, dtype):
    """(device, rows, pointer, pointer of the scales or None, x's dtype code, y's
    dtype)"""
    if isinstance(x, MXTensor):
        device = _device_of(x.codes, "x.codes")
        _check_tensor(x, "x", device, 2)
        if dtype is None:
            dtype = torch.bfloat16 if x.dtype == torch.float32 else x.dtype
        T, xK, data, scales, xt = x.codes.shape[1], x.K, x.codes.data_ptr(), x.scales.data_ptr(), 0
    else:
        xt = _type_of(x, _DTYPES16, "x")
        device = _device_of(x, "x")
        check(x, "x", x.dtype, 2, device)
        if dtype is not None and dtype != x.dtype:
            raise TypeError("the results of 16-bit activations have their type")
        dtype, (T, xK), data, scales = x.dtype, x.shape, x.data_ptr(), None
    if xK != K:
        raise ValueError(f"x has K={xK}, the weight K={K}")
    return device, T, data, scales, xt, dtype


def kernel(R: int, N: int, K: int, quantized: bool, experts: Optional[int] = None):
    """The kernel that gemm() runs for R rows, or grouped_gemm() over `experts`
    (pure host): ("small", row tiles, column tiles, waves along K) or ("large",
    output tile, parts of K)."""
    form = (ctypes.c_int32 * 4)()
    _raise(_mx().w4a16_mx_kernel(R, experts or 1, N, K, quantized, experts is not None, form), "w4a16_mx_kernel")
    tiles = ("64x128", "64x256", "128x128", "128x256", "256x256")
    return ("large", tiles[form[1]], form[2]) if form[0] else ("small", *form[1:])


@functools.lru_cache(maxsize=4096)
def gemm_workspace_size(M: int, N: int, K: int, quantized: bool) -> int:
    b = ctypes.c_size_t()
    _raise(_mx().w4a16_mx_gemm_workspace_size(M, N, K, quantized, ctypes.byref(b)), "w4a16_mx_gemm_workspace_size")
    return b.value


def gemm(x, w: MXWeight, out: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [M, N] = x [M, K] . dequantize(w)^T, with fp32 sums.

    x: fp16 or bf16, whose type Y has; the weights enter as their values in
    that type (in fp16: subnormal below 2^-14, infinite from 65520 on).  Or an
    MXTensor: both operands enter as they are, and Y has `dtype` (if None,
    x.dtype, of an fp32 one bf16).  M may be 0.

    workspace: at least gemm_workspace_size() bytes, for callers that manage
    their own; without one, a call that needs it takes a new block of torch's
    allocator (so calls on other streams, and captured ones, have their own)."""
    if not isinstance(w, MXWeight):
        raise TypeError("w must be an MXWeight")
    device, M, data, scales, xt, dtype = _activations(x, w.K, dtype)
    yt = _float_type(dtype, _DTYPES16, "dtype")
    _check_weight(w, device)
    if w.E != 1:
        raise ValueError("a weight of several experts goes to grouped_gemm")
    if out is None:
        out = torch.empty((M, w.N), dtype=dtype, device=w.q.device)
    else:
        check(out, "out", dtype, 2, device)
        if tuple(out.shape) != (M, w.N):
            raise ValueError("out must be [M, N]")
    stream = stream_of(device)
    if not M:
        return out
    ws, wsb = None, 0
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the call's device")
        ws, wsb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        wsb = gemm_workspace_size(M, w.N, w.K, scales is not None)
        if wsb:
            workspace = w.q.new_empty(wsb)
            ws = workspace.data_ptr()
    _raise(_mx().w4a16_mx_gemm(data, scales, xt, M, w.K, w.q.data_ptr(), w.s.data_ptr(), w.N, yt, out.data_ptr(),
                               ws, wsb, stream), "w4a16_mx_gemm")
    return out


def grouped_gemm(x, w: MXWeight, offsets: torch.Tensor, rows: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Y [R, N]: Y[i] = x[rows[i]] . dequantize(w_e)^T for offsets[e] <= i <
    offsets[e + 1], the rows of expert e; without rows, Y[i] = x[i] . ...

    x [T, K] as gemm()'s, offsets int32 [E + 1], rising from 0 or more to R or
    less, rows int32 [R] (a row whose index lies outside 0..T-1 counts as
    zeros).  An expert may have no rows.  Rows of Y that no expert has stay as they
    are in `out`, and are undefined without one.  R may be 0."""
    if not isinstance(w, MXWeight):
        raise TypeError("w must be an MXWeight")
    device, T, data, scales, xt, dtype = _activations(x, w.K, dtype)
    yt = _float_type(dtype, _DTYPES16, "dtype")
    _check_weight(w, device)
    check(offsets, "offsets", torch.int32, 1, device)
    if offsets.shape[0] != w.E + 1:
        raise ValueError("offsets must be [E + 1]")
    R = T
    if rows is not None:
        check(rows, "rows", torch.int32, 1, device)
        R = rows.shape[0]
    if out is None:
        out = torch.empty((R, w.N), dtype=dtype, device=w.q.device)
    else:
        check(out, "out", dtype, 2, device)
        if tuple(out.shape) != (R, w.N):
            raise ValueError("out must be [R, N]")
    stream = stream_of(device)
    if not R:
        return out
    if not T:
        raise ValueError("x has no rows")
    _raise(_mx().w4a16_mx_grouped_gemm(
        data, scales, xt, T, w.K, None if rows is None else rows.data_ptr(), R, offsets.data_ptr(), w.E,
        w.q.data_ptr(), w.s.data_ptr(), w.N, yt, out.data_ptr(), stream), "w4a16_mx_grouped_gemm")
    return out
