"""Experts over int4 weights: routing, the experts' products, and a layer.

    logits [T, E]                        -> route()   -> ids int32 [T, k], weights fp32 [T, k]
    codes uint8 [E, N, K], scales, zeros -> expert_weight() -> ExpertWeight (device layout)
    X [T, K], ids, weights, gate_up, down -> experts() -> Y [T, D]

A thin binding over libw4a16.so (C ABI in include/w4a16_routed.h): arguments
are checked and marshalled here, every step runs in the library's HIP kernels
on the current stream.  Serving only: no gradients are formed.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import (BF16, PARTIAL_LAST_GROUP, SYMMETRIC, _need, _need16, _raise, lib, pack,
               repack, repack_size)

MAX_EXPERTS = 1024
MAX_K = 32

# Symbols of include/w4a16_routed.h bound here.
EXPORTS = ("w4a16_route", "w4a16_check_route_args", "w4a16_experts_workspace_size",
           "w4a16_experts", "w4a16_check_experts_args")

_ROUTE_SIGMOID, _ROUTE_RENORMALIZE = 0x1, 0x2
_LOGITS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}

_bound = None


def _routed():
    """libw4a16.so with this module's argument types set."""
    global _bound
    if _bound is None:
        L = lib()
        P, I64, I32, U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
        F, SZ = ctypes.c_float, ctypes.c_size_t
        route = [P, I32, I64, I64, P, I32, I32, I32, I32, F, U32, P, P]
        L.w4a16_check_route_args.argtypes = route
        L.w4a16_route.argtypes = route + [P]
        L.w4a16_experts_workspace_size.argtypes = [I64, I32, I64, I64, I64, I64, I32, U32,
                                                   ctypes.POINTER(SZ)]
        experts = [P, I64, I64, P, P, I32, I64, P, P, P, I64, P, P, P, I64, I32, U32, P, P, SZ]
        L.w4a16_check_experts_args.argtypes = experts
        L.w4a16_experts.argtypes = experts + [P]
        for name in EXPORTS:
            getattr(L, name).restype = I32
        _bound = L
    return _bound


def check(t, name: str, dtype, ndim: int, device: int) -> None:
    """_need() for a tensor that must be on the call's device: one small
    function, since a decode step's calls are made of its cost."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device} like the call's first tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def stream_of(device: int) -> int:
    """The current stream of the current device, which must be `device`: the
    kernels are enqueued on it."""
    if device != torch.cuda.current_device():
        raise ValueError(f"tensors on cuda:{device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(device)


def device_layout_bytes(N: int, K: int, g: int):
    """Bytes of q, s and z of one [N, K] matrix in the device layout
    (repack_size() without its checks, which the call itself makes)."""
    nt, G = (N + 15) // 16, -(-K // g)
    return nt * ((K + 127) // 128) * 1024, nt * G * 32, nt * ((G + 7) // 8) * 64


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def route(logits: torch.Tensor, k: int, score: str = "softmax",
          bias: Optional[torch.Tensor] = None, groups: int = 1, topk_groups: int = 1,
          group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
    """Chooses k of E experts for each row of logits [T, E] (fp16, bf16 or
    fp32) -> (ids int32 [T, k], weights fp32 [T, k]), largest first, of equal
    experts the lowest index.

    score: "softmax" over the row or "sigmoid".  bias (fp32 [E]) is added to
    the scores to choose, not to weigh.  With groups > 1, only the experts of
    the topk_groups best of the groups of E / groups consecutive experts are
    left, a group being worth the sum of its group_top (1 or 2) best.
    renormalize divides a row's weights by their sum; scale multiplies them.

    A logit of -inf or NaN (or a bias of -inf or NaN) excludes an expert; a
    slot that no expert is left for has id -1 and weight 0, which experts()
    skips.  T may be 0."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _LOGITS:
        raise TypeError("logits must be a float16, bfloat16 or float32 tensor")
    _need(logits, "logits", logits.dtype, 2)
    device = logits.get_device()
    if score not in ("softmax", "sigmoid"):
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    if not 0 < k <= MAX_K:   # (before memory is taken for it)
        raise ValueError(f"k must be 1 to {MAX_K}")
    T, E = logits.shape
    if bias is not None:
        check(bias, "bias", torch.float32, 1, device)
        if bias.shape[0] != E:
            raise ValueError("bias must be [E]")
    stream = stream_of(device)
    # (the library's checks hold for the empty call too)
    if T == 0:
        _raise(_routed().w4a16_check_route_args(16, _LOGITS[logits.dtype], 1, E, _at(bias), k,
                                                groups, topk_groups, group_top, scale, 0, 16, 16),
               "w4a16_route")
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    if T:
        flags = (_ROUTE_SIGMOID if score == "sigmoid" else 0) | (_ROUTE_RENORMALIZE if renormalize else 0)
        _raise(_routed().w4a16_route(logits.data_ptr(), _LOGITS[logits.dtype], T, E, _at(bias), k,
                                     groups, topk_groups, group_top, scale, flags, ids.data_ptr(),
                                     weights.data_ptr(), stream), "w4a16_route")
    return ids, weights


@dataclass
class ExpertWeight:
    """The weights of E experts in the device layout, one repack() result
    after the other (gated: gate and up of each expert), owned by torch
    tensors.  N counts the rows of one matrix."""
    q: torch.Tensor
    s: torch.Tensor
    z: Optional[torch.Tensor]
    E: int
    N: int
    K: int
    g: int
    flags: int
    gated: bool


def expert_weight(codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor],
                  g: int = 128, gated: bool = False) -> ExpertWeight:
    """codes uint8 [E, N, K] (0..15), scales fp16 or bf16 [E, N, G], zeros uint8
    [E, N, G] or None (symmetric), on the device -> ExpertWeight.  gated: rows
    0 .. N/2 - 1 of an expert are its gate projection, the others up.  K not a
    multiple of g has a partial last group."""
    _need(codes, "codes", torch.uint8, 3)
    bf = _need16(scales, "scales", 3)
    device = codes.get_device()
    check(scales, "scales", scales.dtype, 3, device)
    if g < 1:
        raise ValueError("g must be 32, 64, 128 or 256")
    E, N, K = codes.shape
    G = -(-K // g)
    if tuple(scales.shape) != (E, N, G):
        raise ValueError("scales must be [E, N, ceil(K/g)]")
    if zeros is not None:
        check(zeros, "zeros", torch.uint8, 3, device)
        if tuple(zeros.shape) != (E, N, G):
            raise ValueError("zeros must be [E, N, ceil(K/g)]")
    if E < 1 or E > MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts")
    parts = 2 if gated else 1
    if N % parts:
        raise ValueError("a gated weight has an even number of rows")
    stream_of(device)
    n, m = N // parts, E * parts
    flags = (SYMMETRIC if zeros is None else 0) | (PARTIAL_LAST_GROUP if K % g else 0) | (BF16 if bf else 0)
    repack_size(n, K, g, flags)   # one matrix's own limits
    pad = -n % 16

    def whole_tiles(t, j0, j1):
        """Matrices j0 .. j1 - 1 one below the other, each with rows of zeros up
        to a whole row tile: repack()ed together, they are laid out as one by one."""
        t = t.reshape(m, n, -1)[j0:j1]
        if pad:
            t = torch.nn.functional.pad(t, (0, 0, 0, pad))
        return t.reshape((j1 - j0) * (n + pad), -1)

    # as many matrices at once as repack() takes rows and weights
    step = max(1, min(m, (1 << 26) // (n + pad), (1 << 34) // ((n + pad) * K)))
    done = []
    for j0 in range(0, m, step):
        j1 = min(m, j0 + step)
        rows = whole_tiles(scales, j0, j1)
        if rows.data_ptr() % 16:
            rows = rows.clone()
        done.append(repack(pack(whole_tiles(codes, j0, j1)), rows,
                           None if zeros is None else pack(whole_tiles(zeros, j0, j1)), K, g,
                           symmetric=zeros is None, partial=K % g != 0))
    if len(done) == 1:
        q, s, z = done[0].q, done[0].s, done[0].z
    else:
        q, s = torch.cat([w.q for w in done]), torch.cat([w.s for w in done])
        z = None if zeros is None else torch.cat([w.z for w in done])
    return ExpertWeight(q, s, z, E, n, K, g, flags, gated)


def _check_expert_weight(w: ExpertWeight, name: str, device: int) -> None:
    """The device-layout tensors hold the bytes the shape needs (the kernels
    read them through bare pointers)."""
    qb, sb, zb = device_layout_bytes(w.N, w.K, w.g)
    m = w.E * (2 if w.gated else 1)
    check(w.q, name, torch.uint8, w.q.dim(), device)
    check(w.s, name, torch.bfloat16 if w.flags & BF16 else torch.float16, w.s.dim(), device)
    small = w.q.numel() < m * qb or w.s.numel() * 2 < m * sb
    if not w.flags & SYMMETRIC:
        check(w.z, name, torch.int32, w.z.dim(), device)
        small = small or w.z.numel() * 4 < m * zb
    if small:
        raise ValueError(f"{name} tensors are smaller than its shape needs")


def experts_workspace_size(T: int, k: int, gate_up: ExpertWeight, down: ExpertWeight) -> int:
    b = ctypes.c_size_t()
    _raise(_routed().w4a16_experts_workspace_size(T, k, gate_up.K, gate_up.N, down.N, gate_up.E,
                                                  gate_up.g, gate_up.flags | down.flags,
                                                  ctypes.byref(b)),
           "w4a16_experts_workspace_size")
    return b.value


def experts(X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up: ExpertWeight,
            down: ExpertWeight, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [T, D]: Y[t] = sum over the slots j of weights[t, j] * h . Wdown_e^T,
    h = silu(X[t] . Wgate_e^T) * (X[t] . Wup_e^T), e = ids[t, j].

    X [T, K] fp16 or bf16 (the weights' format), ids int32 [T, k] and weights
    fp32 [T, k] as route() gives them.  A slot with an id outside 0..E-1 adds
    nothing; a row with no other slot is 0.  T may be 0.  fp16: a row whose h
    leaves the type's range somewhere is still right, but slow.

    workspace: at least experts_workspace_size() bytes, for callers that
    manage their own; without one, each call takes a new block of torch's
    allocator (so calls on other streams, and captured ones, have their own)."""
    bf = _need16(X, "X", 2)
    device = X.get_device()
    check(ids, "ids", torch.int32, 2, device)
    check(weights, "weights", torch.float32, 2, device)
    T, K = X.shape
    if not gate_up.gated or down.gated:
        raise ValueError("gate_up must be a gated ExpertWeight and down a plain one")
    if gate_up.E != down.E or gate_up.N != down.K or gate_up.g != down.g or K != gate_up.K:
        raise ValueError(f"X [T, {K}], gate_up [{gate_up.E}, 2 x {gate_up.N}, {gate_up.K}] and down "
                         f"[{down.E}, {down.N}, {down.K}] do not fit (group sizes {gate_up.g}, {down.g})")
    if (gate_up.flags ^ down.flags) & (SYMMETRIC | BF16) or bf != bool(gate_up.flags & BF16):
        raise TypeError("X, gate_up and down must share a 16-bit format, and the weights symmetry")
    k = ids.shape[1]
    if ids.shape[0] != T or weights.shape != ids.shape:
        raise ValueError("ids and weights must be [T, k]")
    _check_expert_weight(gate_up, "gate_up", device)
    _check_expert_weight(down, "down", device)
    if out is None:
        out = X.new_empty((T, down.N))
    else:
        check(out, "out", X.dtype, 2, device)
        if tuple(out.shape) != (T, down.N):
            raise ValueError("out must be [T, D]")
    stream = stream_of(device)
    need = experts_workspace_size(max(T, 1), k, gate_up, down)
    if T == 0:
        return out
    if workspace is None:
        workspace = ids.new_empty(need // 4)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the call's device")
    _raise(_routed().w4a16_experts(
        X.data_ptr(), T, K, ids.data_ptr(), weights.data_ptr(), k, gate_up.E, gate_up.q.data_ptr(),
        gate_up.s.data_ptr(), _at(gate_up.z), gate_up.N, down.q.data_ptr(), down.s.data_ptr(),
        _at(down.z), down.N, gate_up.g, gate_up.flags | down.flags, out.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), stream), "w4a16_experts")
    return out


class QExperts(torch.nn.Module):
    """A layer of E gated experts over int4 weights: y = experts(x, route(logits)).

    gate_up and down are expert_weight() results; the other arguments are
    route()'s.  forward takes x [..., K] and the router's logits [..., E]."""

    def __init__(self, gate_up: ExpertWeight, down: ExpertWeight, k: int, score: str = "softmax",
                 bias: Optional[torch.Tensor] = None, groups: int = 1, topk_groups: int = 1,
                 group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
        super().__init__()
        self.gate_up, self.down = gate_up, down
        self.routing = dict(k=k, score=score, bias=bias, groups=groups, topk_groups=topk_groups,
                            group_top=group_top, renormalize=renormalize, scale=scale)

    def forward(self, x: torch.Tensor, logits: torch.Tensor,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        if (x.shape[:-1] != logits.shape[:-1] or x.shape[-1:] != (self.gate_up.K,)
                or logits.shape[-1:] != (self.gate_up.E,)):
            raise ValueError(f"x must be [..., {self.gate_up.K}] and logits [..., {self.gate_up.E}] with the "
                             f"same leading dimensions, got {tuple(x.shape)} and {tuple(logits.shape)}")
        ids, weights = route(logits.reshape(-1, self.gate_up.E), **self.routing)
        y = experts(x.reshape(-1, self.gate_up.K), ids, weights, self.gate_up, self.down, out=out)
        return y.reshape(*x.shape[:-1], self.down.N)
