"""Low-rank adapters of many requests at once beside a shared int4 projection.

    A [n, parts, r, K], B [n, N, r], scales [n] -> adapters() -> Adapters
    X [M, K], PackedWeight, Adapters, ids [M]   -> gemm_lora() -> Y [M, N]

    Y[m] = X[m] . dequant(W)^T + scales[a] * (X[m] . A_a^T) . B_a^T,   a = ids[m]

A thin binding over libw4a16.so (C ABI in include/w4a16_routed.h).  Serving
only: no gradients are formed.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field
from typing import Optional, Sequence

import torch

from . import (BF16, PATH_LARGE_M, PATH_SMALL_M, PackedWeight, _check_packed, _need, _need16,
               _raise, lib)
from .moe import _at, on_current_device

MAX_PARTS = 8
MAX_RANK = 256

# Symbols of include/w4a16_routed.h bound here.
EXPORTS = ("w4a16_gemm_lora_workspace_size", "w4a16_gemm_lora", "w4a16_check_gemm_lora_args")

_bound = None


def _routed():
    """libw4a16.so with this module's argument types set."""
    global _bound
    if _bound is None:
        L = lib()
        P, I64, I32, U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
        SZ, PI64 = ctypes.c_size_t, ctypes.POINTER(ctypes.c_int64)
        L.w4a16_gemm_lora_workspace_size.argtypes = [I64, I64, I64, I32, U32, I32, I32,
                                                     ctypes.POINTER(SZ)]
        args = [P, I64, I64, P, P, P, I64, I32, U32, P, P, P, I64, I32, I32, PI64, P, P, P, SZ]
        L.w4a16_check_gemm_lora_args.argtypes = args
        L.w4a16_gemm_lora.argtypes = args + [P]
        for name in EXPORTS:
            getattr(L, name).restype = I32
        _bound = L
    return _bound


@dataclass
class Adapters:
    """n low-rank adapters of one projection, owned by torch tensors."""
    A: torch.Tensor        # 16-bit [n, parts * r, K]
    B: torch.Tensor        # 16-bit [n, N, r]
    scales: torch.Tensor   # fp32 [n]
    n: int
    r: int
    sizes: Sequence[int]   # columns of each part
    c_sizes: ctypes.Array = field(repr=False, default=None)

    @property
    def K(self) -> int:
        return self.A.shape[2]

    @property
    def N(self) -> int:
        return self.B.shape[1]


def adapters(A: torch.Tensor, B: torch.Tensor, scales: torch.Tensor,
             sizes: Optional[Sequence[int]] = None) -> Adapters:
    """A [n, parts, r, K] (or [n, r, K] for one part) and B [n, N, r], fp16 or
    bf16, scales fp32 [n], on the device -> Adapters.  sizes: the columns of
    each part (the sizes of a fused projection); part p of the columns uses
    A[:, p].  A rank that is no multiple of 8 is padded with zeros (a copy), and
    adapters of smaller rank may be padded with zeros up to r."""
    bf = _need16(A, "A")
    _need(B, "B", torch.bfloat16 if bf else torch.float16, 3)
    _need(scales, "scales", torch.float32, 1)
    if A.dim() == 3:
        A = A.unsqueeze(1)
    if A.dim() != 4:
        raise ValueError("A must be [n, parts, r, K] or [n, r, K]")
    n, parts, r, K = A.shape
    N = B.shape[1]
    sizes = [N] if sizes is None else [int(s) for s in sizes]
    if len(sizes) != parts or parts < 1 or parts > MAX_PARTS or min(sizes) < 1 or sum(sizes) != N:
        raise ValueError(f"sizes must be the columns of the {parts} parts (at most {MAX_PARTS}), {N} in all")
    if n < 1 or tuple(B.shape) != (n, N, r) or scales.shape[0] != n:
        raise ValueError("B must be [n, N, r] and scales [n]")
    if r < 1 or r > MAX_RANK:
        raise ValueError(f"a rank of 1 to {MAX_RANK}")
    on_current_device(A, B, scales)
    if r % 8:
        pad = 8 - r % 8
        A = torch.cat([A, A.new_zeros((n, parts, pad, K))], 2)
        B = torch.cat([B, B.new_zeros((n, N, pad))], 2)
        r += pad
    return Adapters(A.reshape(n, parts * r, K).contiguous(), B.contiguous(), scales, n, r, sizes,
                    (ctypes.c_int64 * parts)(*sizes))


def gemm_lora_workspace_size(M: int, w: PackedWeight, ad: Adapters, flags: int = 0) -> int:
    b = ctypes.c_size_t()
    _raise(_routed().w4a16_gemm_lora_workspace_size(M, w.N, w.K, w.g, w.flags | flags,
                                                    len(ad.sizes), ad.r, ctypes.byref(b)),
           "w4a16_gemm_lora_workspace_size")
    return b.value


def gemm_lora(X: torch.Tensor, w: PackedWeight, ad: Adapters, ids: torch.Tensor,
              path: Optional[str] = None, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gemm() with an adapter for each row: Y [M, N] as above, X [M, K] fp16 or
    bf16 (the weight's and the adapters' format), ids int32 [M].  A row whose
    id lies outside 0..n-1 (-1 by custom) has no adapter.

    path as gemm()'s.  workspace: at least gemm_lora_workspace_size() bytes, for
    callers that manage their own; without one, each call takes a new block of
    torch's allocator (so calls on other streams, and captured ones, have
    their own)."""
    bf = _need16(X, "X", 2)
    _need(ids, "ids", torch.int32, 1)
    M, K = X.shape
    if K != w.K or w.K != ad.A.shape[2] or w.N != ad.B.shape[1]:
        raise ValueError(f"X has K={K}, the weight is [{w.N}, {w.K}], the adapters [{ad.N}, {ad.K}]")
    if bf != bool(w.flags & BF16) or X.dtype != ad.A.dtype:
        raise TypeError("X, the weight's scales and the adapters must share one 16-bit format")
    if ids.shape[0] != M:
        raise ValueError("ids must be [M]")
    n, pr = ad.n, len(ad.sizes) * ad.r
    if tuple(ad.A.shape) != (n, pr, K) or tuple(ad.B.shape) != (n, w.N, ad.r) or \
            ad.B.dtype != X.dtype or tuple(ad.scales.shape) != (n,) or \
            not (ad.A.is_contiguous() and ad.B.is_contiguous()):
        raise ValueError("the adapters' tensors do not have the shapes they need (use adapters())")
    flags = w.flags
    if path == "small_m":
        flags |= PATH_SMALL_M
    elif path == "large_m":
        flags |= PATH_LARGE_M
    elif path is not None:
        raise ValueError("path must be None, 'small_m' or 'large_m'")
    _check_packed(w)
    if out is None:
        out = torch.empty((M, w.N), dtype=X.dtype, device=X.device)
    else:
        _need(out, "out", X.dtype, 2)
        if tuple(out.shape) != (M, w.N):
            raise ValueError("out must be [M, N]")
    if workspace is None:
        workspace = torch.empty(gemm_lora_workspace_size(M, w, ad, flags), dtype=torch.uint8,
                                device=X.device)
    elif not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous device tensor")
    stream = on_current_device(X, ids, w.q, w.s, w.z, ad.A, ad.B, ad.scales, out, workspace)
    _raise(_routed().w4a16_gemm_lora(
        X.data_ptr(), M, K, w.q.data_ptr(), w.s.data_ptr(), _at(w.z), w.N, w.g, flags,
        ad.A.data_ptr(), ad.B.data_ptr(), ad.scales.data_ptr(), n, ad.r, len(ad.sizes), ad.c_sizes,
        ids.data_ptr(), out.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), stream), "w4a16_gemm_lora")
    return out
