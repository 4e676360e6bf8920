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

from . import (BF16, PATH_LARGE_M, PATH_SMALL_M, SYMMETRIC, PackedWeight, _need, _need16, _raise,
               lib)
from .moe import _at, check, device_layout_bytes, stream_of

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
    c_sizes: ctypes.Array = field(repr=False)   # columns of each part

    @property
    def sizes(self):
        return list(self.c_sizes)

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
    device = A.get_device()
    check(B, "B", torch.bfloat16 if bf else torch.float16, 3, device)
    check(scales, "scales", torch.float32, 1, device)
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
    if r % 8:
        pad = 8 - r % 8
        A = torch.cat([A, A.new_zeros((n, parts, pad, K))], 2)
        B = torch.cat([B, B.new_zeros((n, N, pad))], 2)
        r += pad
    return Adapters(A.reshape(n, parts * r, K).contiguous(), B.contiguous(), scales, n, r,
                    (ctypes.c_int64 * parts)(*sizes))


def gemm_lora_workspace_size(M: int, w: PackedWeight, ad: Adapters, flags: int = 0) -> int:
    b = ctypes.c_size_t()
    _raise(_routed().w4a16_gemm_lora_workspace_size(M, w.N, w.K, w.g, w.flags | flags,
                                                    len(ad.c_sizes), ad.r, ctypes.byref(b)),
           "w4a16_gemm_lora_workspace_size")
    return b.value


def gemm_lora(X: torch.Tensor, w: PackedWeight, ad: Adapters, ids: torch.Tensor,
              path: Optional[str] = None, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gemm() with an adapter for each row: Y [M, N] as above, X [M, K] fp16 or
    bf16 (the weight's and the adapters' format), ids int32 [M].  A row whose
    id lies outside 0..n-1 (-1 by custom) has no adapter.  At least one row, as
    gemm() takes.

    path as gemm()'s.  workspace: at least gemm_lora_workspace_size() bytes, for
    callers that manage their own; without one, each call takes a new block of
    torch's allocator (so calls on other streams, and captured ones, have
    their own)."""
    bf = _need16(X, "X", 2)
    device, dtype = X.get_device(), X.dtype
    check(ids, "ids", torch.int32, 1, device)
    M, K = X.shape
    N = w.N
    if K != w.K or w.K != ad.A.shape[2] or N != ad.B.shape[1]:
        raise ValueError(f"X has K={K}, the weight is [{N}, {w.K}], the adapters [{ad.N}, {ad.K}]")
    if bf != bool(w.flags & BF16):
        raise TypeError("X, the weight's scales and the adapters must share one 16-bit format")
    if ids.shape[0] != M:
        raise ValueError("ids must be [M]")
    n, r, parts = ad.n, ad.r, len(ad.c_sizes)
    check(ad.A, "adapters.A", dtype, 3, device)
    check(ad.B, "adapters.B", dtype, 3, device)
    check(ad.scales, "adapters.scales", torch.float32, 1, device)
    if ad.A.shape != (n, parts * r, K) or ad.B.shape != (n, N, r) or ad.scales.shape[0] != n:
        raise ValueError("the adapters' tensors do not have the shapes they need (use adapters())")
    flags = w.flags
    if path == "small_m":
        flags |= PATH_SMALL_M
    elif path == "large_m":
        flags |= PATH_LARGE_M
    elif path is not None:
        raise ValueError("path must be None, 'small_m' or 'large_m'")
    # the weight's tensors hold the bytes its shape needs
    qb, sb, zb = device_layout_bytes(N, K, w.g)
    check(w.q, "w.q", torch.uint8, w.q.dim(), device)
    check(w.s, "w.s", dtype, w.s.dim(), device)
    small = w.q.numel() < qb or w.s.numel() * 2 < sb
    if not flags & SYMMETRIC:
        check(w.z, "w.z", torch.int32, w.z.dim(), device)
        small = small or w.z.numel() * 4 < zb
    if small:
        raise ValueError("PackedWeight tensors are smaller than its shape needs")
    if out is None:
        out = X.new_empty((M, N))
    else:
        check(out, "out", dtype, 2, device)
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N]")
    stream = stream_of(device)
    if workspace is None:
        workspace = ids.new_empty((gemm_lora_workspace_size(M, w, ad, flags) + 3) // 4)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the call's device")
    _raise(_routed().w4a16_gemm_lora(
        X.data_ptr(), M, K, w.q.data_ptr(), w.s.data_ptr(), _at(w.z), N, w.g, flags,
        ad.A.data_ptr(), ad.B.data_ptr(), ad.scales.data_ptr(), n, r, parts, ad.c_sizes,
        ids.data_ptr(), out.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), stream), "w4a16_gemm_lora")
    return out
