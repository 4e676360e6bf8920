"""Plain definitions of the routed operators in 64 bits (torch on the CPU),
with a bound of what a computation with 32-bit sums and the operators' stated
roundings may differ by.  Shares no code with the GPU path.

u16 is half a step of the 16-bit type relative to a value (torch.finfo(t).eps
/ 2); a 32-bit sum of n products in any order, started anew per group or not,
is off by at most 2 n 2^-24 of the sum of their absolute values (n roundings
of the products and n of the sums).
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24


def weight(codes, scales, zeros, g):
    """RNE16((q - z) s) in 64 bits; codes [..., N, K], scales and zeros [..., N, G].
    (The product is exact in 64 bits, so it is rounded once.)"""
    K = codes.shape[-1]
    grp = torch.arange(K) // g
    z = torch.full_like(scales, 8, dtype=torch.float64) if zeros is None else zeros.double()
    w = (codes.double() - z[..., grp]) * scales.double()[..., grp]
    return w.to(scales.dtype).double()


def route(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1,
          renormalize=True, scale=1.0):
    """(ids, weights, bound): by sorting whole rows in 64 bits.

    Bound: a score's exponent l - max is rounded to 32 bits (2^-24 |l - max|
    in the exponential's argument), the exponential is good to 2 steps, and
    the quotient, the sums and the scale add a handful of roundings, E of
    them in a softmax's sum."""
    l = logits.double()
    l = torch.where(torch.isnan(l), -torch.inf, l).clamp(max=torch.finfo(torch.float32).max)
    T, E = l.shape
    dead = torch.isinf(l)
    top = l.max(1, keepdim=True).values
    top = torch.where(torch.isinf(top), 0.0, top)
    if score == "softmax":
        s = torch.exp(l - top)
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
        arg = (l - top).abs()
    else:
        s = 1 / (1 + torch.exp(-l))
        arg = torch.zeros_like(l)
    s = torch.where(dead, 0.0, s)
    # without a bias the order of the scores is that of the logits, whose
    # neighbours a 64-bit exponential may no longer tell apart
    raw = bias is None and not (topk_groups < groups and group_top == 2)
    key = l.clone() if raw else s.clone()
    if bias is not None:
        key = key + bias.double()
        dead = dead | torch.isnan(key) | (key == -torch.inf)
    key = torch.where(dead, -torch.inf, key)
    if topk_groups < groups:
        per = key.reshape(T, groups, -1)
        best = per.sort(dim=2, descending=True).values[:, :, :group_top]
        value = torch.where(torch.isinf(best) & (best < 0), 0.0, best).sum(2)
        value = torch.where(best[:, :, 0] == -torch.inf, -torch.inf, value)
        chosen = value.sort(dim=1, descending=True, stable=True).indices[:, :topk_groups]
        keep = torch.zeros((T, groups), dtype=torch.bool).scatter_(1, chosen, True)
        key = torch.where(keep.repeat_interleave(E // groups, 1), key, -torch.inf)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    none = key.gather(1, ids) == -torch.inf
    w = torch.where(none, 0.0, s.gather(1, ids))
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = w * scale
    far = arg.gather(1, ids)
    far = torch.where(torch.isinf(far), 0.0, far).max(1, keepdim=True).values
    bound = w.abs() * U32 * (2 * far + E + 16) + 1e-38
    return torch.where(none, -1, ids).to(torch.int32), w, bound


def experts(X, ids, weights, gate_up, down, g):
    """(Y, bound).  gate_up = (codes [E, 2I, K], scales, zeros), down = (codes
    [E, D, I], scales, zeros).

    Bound: gate and up are 32-bit sums of K products; silu's slope is at most
    1.1 and its own arithmetic, v / (1 + exp(-v)) with exp2's argument and each
    of the exponential, sum, quotient and product rounded, is off by at most
    (2 |v| + 8) 2^-24 of it; h is rounded to 16 bits (or to the smallest
    subnormal's half); the down product adds I products, the weighted sum k;
    the result is rounded to 16 bits."""
    dt = X.dtype
    u, tiny = torch.finfo(dt).eps / 2, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    Xd, E = X.double(), gate_up[0].shape[0]
    T, k = ids.shape
    I, D, K = gate_up[0].shape[1] // 2, down[0].shape[1], X.shape[1]
    Y = torch.zeros((T, D), dtype=torch.float64)
    err = torch.zeros((T, D), dtype=torch.float64)
    mag = torch.zeros((T, D), dtype=torch.float64)
    for e in range(E):
        at = (ids == e).nonzero()
        if not len(at):
            continue
        rows, wt = at[:, 0], weights[at[:, 0], at[:, 1]].double()[:, None]
        Wg = weight(*[t if t is None else t[e] for t in gate_up], g)
        Wd = weight(*[t if t is None else t[e] for t in down], g)
        x = Xd[rows]
        gu, gua = x @ Wg.T, x.abs() @ Wg.abs().T
        gate, up = gu[:, :I], gu[:, I:]
        eg, eu = 2 * K * U32 * gua[:, :I], 2 * K * U32 * gua[:, I:]
        sl = gate * torch.special.expit(gate)
        h = sl * up
        es = 1.1 * eg + (2 * gate.abs() + 8) * U32 * sl.abs()
        eh = es * up.abs() + (sl.abs() + es) * eu
        eh = eh + u * (h.abs() + eh) + tiny
        out = h @ Wd.T
        e_out = eh @ Wd.abs().T + 2 * I * U32 * ((h.abs() + eh) @ Wd.abs().T)
        Y.index_add_(0, rows, wt * out)
        err.index_add_(0, rows, wt.abs() * e_out)
        mag.index_add_(0, rows, wt.abs() * (out.abs() + e_out))
    err = err + 2 * (k + 1) * U32 * mag
    return Y, err + u * (Y.abs() + err) + tiny


def gemm_lora(X, W, A, B, scales, ids, sizes):
    """(Y, bound).  W (codes, scales, zeros, g); A [n, parts, r, K], B [n, N, r].

    Bound: the projection is a 32-bit sum of K products whose weights may be
    unrounded (half a 16-bit step of each); the low-rank values are 32-bit sums
    of K products, and enter a sum of r products as 16 significant bits (2^-16
    of each product; in fp16 22 bits of the largest of a row's 32 ranks, which
    is 2^-22 of the sum of all of them)."""
    dt = X.dtype
    u, tiny = torch.finfo(dt).eps / 2, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    Xd, K = X.double(), X.shape[1]
    Wd = weight(*W)
    Y = Xd @ Wd.T
    err = (u + 2 * (K + 2) * U32) * (Xd.abs() @ Wd.abs().T)
    n, parts, r, _ = A.shape
    for a in range(n):
        rows = (ids == a).nonzero()[:, 0]
        if not len(rows):
            continue
        c0 = 0
        for p in range(parts):
            c1 = c0 + sizes[p]
            Ap, Bp = A[a, p].double(), B[a, c0:c1].double()
            s, sa = Xd[rows] @ Ap.T, Xd[rows].abs() @ Ap.abs().T
            es = 2 * (K + 2) * U32 * sa
            sc = scales[a].double()
            Y[rows, c0:c1] += sc * (s @ Bp.T)
            err[rows, c0:c1] += sc.abs() * (es @ Bp.abs().T +
                                            (3 * 2.0 ** -16 + 4 * r * U32) * ((s.abs() + es) @ Bp.abs().T) +
                                            2.0 ** -21 * (s.abs() + es).amax(1, keepdim=True) * Bp.abs().sum(1))
            c0 = c1
    err = err + 2 * U32 * (Y.abs() + err)
    return Y, err + u * (Y.abs() + err) + tiny
