"""Plain definitions of the microscaled 4-bit operators in 64 bits (torch on
the CPU), with a bound of what a computation with 32-bit sums and one rounding
to the result's type may differ by.  Shares no code with the GPU path.
"""
from __future__ import annotations

import torch

BLOCK = 32
SIZES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
U32 = 2.0 ** -24


def quantize(x):
    """x [.., K] -> (element codes uint8 [.., K], scale bytes uint8 [.., blocks]),
    by the distance to each of the eight sizes."""
    K = x.shape[-1]
    v = torch.nn.functional.pad(x.double(), (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    bad = ~torch.isfinite(v).all(-1, keepdim=True)
    v = torch.where(bad, 0.0, v)
    a = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(a).exponent - 3).clamp(-127, 127)     # a = m 2^k, m in [1/2, 1)
    e = torch.where(a == 0, -127, e)
    r = v * torch.exp2(-e.double())                        # exact: a power of two
    far = (r.abs().unsqueeze(-1) - SIZES).abs()
    near = far.amin(-1, keepdim=True)
    # of two sizes equally near, the even number
    key = torch.where(far == near, torch.arange(8) % 2, 9)
    code = key.argmin(-1)
    code = (code + 8 * torch.signbit(v)).to(torch.uint8)
    code = torch.where(bad, 0, code).flatten(-2)[..., :K].to(torch.uint8)
    scale = torch.where(bad, 255, e + 127).squeeze(-1).to(torch.uint8)
    return code, scale


def values(code, scale):
    """Element codes [.., K] and scale bytes -> values in 64 bits."""
    K = code.shape[-1]
    v = SIZES[(code & 7).long()] * torch.where(code >= 8, -1.0, 1.0)
    s = torch.where(scale == 255, torch.nan, torch.exp2(scale.double() - 127))
    return v * s[..., torch.arange(K) // BLOCK]


def pack(code):
    """Two columns a byte, the first in the low half."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def product(X, W, out_dtype):
    """(X W^T in 64 bits, bound): X [M, K] and W [N, K] hold the operands' values.
    A sum of K products in 32 bits, in any order, is off by at most 2 K 2^-24 of
    the sum of their magnitudes (K roundings of products, K of sums); the
    result is rounded to out_dtype once, by half a step of it or of the type's
    smallest number."""
    y = X @ W.T
    info = torch.finfo(out_dtype)
    y32 = 2 * X.shape[1] * U32 * (X.abs() @ W.abs().T)
    return y, y32 * (1 + info.eps) + info.eps / 2 * y.abs() + info.smallest_normal * info.eps / 2


def grouped(X, W, offsets, rows, out_dtype):
    """(Y, bound, written): W [E, N, K]; rows of Y that no expert has are False in
    `written`."""
    R = X.shape[0] if rows is None else rows.shape[0]
    Y = torch.zeros((R, W.shape[1]), dtype=torch.float64)
    bound, written = torch.zeros_like(Y), torch.zeros(R, dtype=torch.bool)
    for e in range(W.shape[0]):
        for i in range(int(offsets[e]), int(offsets[e + 1])):
            j = i if rows is None else int(rows[i])
            x = X[j:j + 1] if 0 <= j < X.shape[0] else torch.zeros_like(X[:1])
            y, b = product(x, W[e], out_dtype)
            Y[i], bound[i], written[i] = y[0], b[0], True
    return Y, bound, written
