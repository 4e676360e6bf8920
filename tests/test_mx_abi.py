"""The microscaled 4-bit operators without a GPU: every symbol their header
declares resolves, and every refusal is a status of the pure-host checks or an
error of the binding."""
import ctypes
import os
import re

import pytest
import torch

import weight_only_int4_02_amd as w4
from oracle import mx as ref
from weight_only_int4_02_amd import mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w4a16_mx.h")
A = 1 << 40


def P(off=0):
    return A + off


def test_every_declared_symbol_resolves():
    names = set(re.findall(r"^int32_t\s+(w4a16_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(mx.EXPORTS)
    h = ctypes.CDLL(w4.LIB_PATH)
    for n in names:
        assert ctypes.cast(getattr(h, n), ctypes.c_void_p).value


def quantize(**kw):
    a = dict(X=P(), dtype=0, M=4, K=64, codes=P(1 << 30), scales=P(1 << 31))
    a.update(kw)
    return mx._mx().w4a16_mx_check_quantize_args(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(), w4.OK), (dict(dtype=2), w4.OK), (dict(K=8), w4.OK),
    (dict(X=None), w4.ERR_NULL), (dict(codes=None), w4.ERR_NULL), (dict(scales=None), w4.ERR_NULL),
    (dict(dtype=3), w4.ERR_SHAPE), (dict(dtype=-1), w4.ERR_SHAPE), (dict(M=0), w4.ERR_SHAPE),
    (dict(K=0), w4.ERR_SHAPE), (dict(K=12), w4.ERR_SHAPE), (dict(K=(1 << 24) + 8), w4.ERR_SHAPE),
    (dict(M=1 << 31, K=8), w4.ERR_SHAPE), (dict(M=1 << 20, K=1 << 18), w4.ERR_SHAPE),
    (dict(X=P(8)), w4.ERR_ALIGN), (dict(codes=P(8)), w4.ERR_ALIGN), (dict(scales=P(4)), w4.ERR_ALIGN),
])
def test_quantize_args(kw, status):
    assert quantize(**kw) == status
    a = dict(X=P(), dtype=0, M=4, K=64, codes=P(1 << 30), scales=P(1 << 31))
    a.update(kw)
    assert mx._mx().w4a16_mx_check_dequantize_args(a["codes"], a["scales"], a["M"], a["K"], a["dtype"], a["X"]) == status


def weight(**kw):
    a = dict(codes=P(), scales=P(), E=2, N=40, K=64, q=P(), s=P())
    a.update(kw)
    return mx._mx().w4a16_mx_check_weight_args(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(), w4.OK), (dict(E=1024), w4.OK), (dict(codes=None), w4.ERR_NULL),
    (dict(s=None), w4.ERR_NULL), (dict(E=0), w4.ERR_SHAPE), (dict(E=1025), w4.ERR_SHAPE), (dict(N=0), w4.ERR_SHAPE),
    (dict(N=1 << 22), w4.ERR_SHAPE), (dict(K=20), w4.ERR_SHAPE), (dict(K=(1 << 20) + 8), w4.ERR_SHAPE),
    (dict(N=1 << 16, K=1 << 16), w4.ERR_SHAPE),     # 2 GiB of codes
    (dict(q=P(4)), w4.ERR_ALIGN), (dict(codes=P(4)), w4.ERR_ALIGN), (dict(scales=P(8)), w4.ERR_ALIGN),
])
def test_weight_args(kw, status):
    assert weight(**kw) == status


def test_weight_size():
    assert mx.weight_size(1, 16, 128) == (1024, 256)
    assert mx.weight_size(3, 17, 640) == (3 * 2 * 5 * 1024, 3 * 2 * 2 * 256)
    with pytest.raises(w4.W4A16ArgumentError):
        mx.weight_size(1, 16, 12)


def gemm(**kw):
    a = dict(X=P(), xs=None, xt=0, M=4, K=64, q=P(1 << 33), s=P(1 << 34), N=40, yt=0, Y=P(1 << 32), ws=P(1 << 37),
             wsb=1 << 40)
    a.update(kw)
    return mx._mx().w4a16_mx_check_gemm_args(*a.values())


PRODUCT = [
    (dict(), w4.OK), (dict(xt=1, yt=1), w4.OK), (dict(xs=P(1 << 31), xt=0, yt=1), w4.OK),
    (dict(X=None), w4.ERR_NULL), (dict(q=None), w4.ERR_NULL), (dict(s=None), w4.ERR_NULL), (dict(Y=None), w4.ERR_NULL),
    (dict(xt=0, yt=1), w4.ERR_SHAPE), (dict(xt=2, yt=2), w4.ERR_SHAPE), (dict(K=4), w4.ERR_SHAPE),
    (dict(N=0), w4.ERR_SHAPE), (dict(X=P(8)), w4.ERR_ALIGN), (dict(Y=P((1 << 32) + 2)), w4.ERR_ALIGN),
    (dict(xs=P(8)), w4.ERR_ALIGN), (dict(q=P(4)), w4.ERR_ALIGN),
    (dict(Y=P(256)), w4.ERR_SHAPE),                      # inside X
    (dict(Y=P(), X=P(0x10000), xs=P(0x100)), w4.ERR_SHAPE),   # over the scales
]


@pytest.mark.parametrize("kw,status", PRODUCT + [
    (dict(M=0), w4.ERR_SHAPE), (dict(M=1 << 31), w4.ERR_SHAPE),
    (dict(M=1 << 18, K=4096), w4.ERR_SHAPE),             # X of 2 GiB
    (dict(M=1 << 18, K=4096, xs=P(1 << 31), N=8), w4.OK)])
def test_gemm_args(kw, status):
    assert gemm(**kw) == status


def grouped(**kw):
    a = dict(X=P(), xs=None, xt=0, T=4, K=64, rows=None, R=4, offsets=P(1 << 35), E=3, q=P(1 << 33), s=P(1 << 34),
             N=40, yt=0, Y=P(1 << 32))
    a.update(kw)
    return mx._mx().w4a16_mx_check_grouped_gemm_args(*a.values())


@pytest.mark.parametrize("kw,status", PRODUCT + [
    (dict(T=5), w4.ERR_SHAPE), (dict(T=5, rows=P(1 << 36)), w4.OK), (dict(R=0), w4.ERR_SHAPE), (dict(T=0), w4.ERR_SHAPE),
    (dict(E=1025), w4.ERR_SHAPE), (dict(offsets=None), w4.ERR_NULL), (dict(offsets=P(2)), w4.ERR_ALIGN),
    (dict(rows=P(2)), w4.ERR_ALIGN), (dict(rows=P((1 << 32) + 8)), w4.ERR_SHAPE),
    (dict(offsets=P((1 << 32) + 8)), w4.ERR_SHAPE)])
def test_grouped_args(kw, status):
    assert grouped(**kw) == status


@pytest.mark.parametrize("kw", [
    dict(codes=P(0x1100)), dict(scales=P(0x1000)), dict(dtype=2, M=64, codes=P(0x4000)),
    dict(codes=P(1 << 31)), dict(scales=P((1 << 30) + 512))])
def test_quantize_overlaps(kw):
    assert quantize(X=P(0x1000), **kw) == w4.ERR_SHAPE


def test_the_workspace_overlaps_nothing():
    shape = dict(M=61, K=11008, N=64)
    need = mx.gemm_workspace_size(61, 64, 11008, False)
    assert need > 0
    assert gemm(**shape) == w4.OK
    assert gemm(**shape, wsb=need) == w4.OK
    assert gemm(**shape, wsb=need - 1) == w4.ERR_WORKSPACE
    assert gemm(**shape, ws=None) == w4.ERR_NULL
    assert gemm(**shape, ws=P((1 << 37) + 8)) == w4.ERR_ALIGN
    for ws in (P((1 << 32) + 61 * 64 * 2 - 16), P((1 << 32) - need + 16), P()):      # Y's end and start, X
        assert gemm(**shape, ws=ws) == w4.ERR_SHAPE
    quantized = dict(M=61, K=11008, N=64, xs=P(1 << 31))
    assert mx.gemm_workspace_size(61, 64, 11008, True) > 0
    assert gemm(**quantized) == w4.OK
    assert gemm(**quantized, ws=P((1 << 31) + 256)) == w4.ERR_SHAPE


def test_the_binding_refuses_what_is_not_on_a_device():
    x = torch.zeros((2, 64), dtype=torch.float16)
    t = mx.MXTensor(torch.zeros((4, 2, 64), dtype=torch.uint8), torch.zeros((1, 2, 16), dtype=torch.uint8), 64)
    w = mx.MXWeight(torch.zeros(1024, dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8), 1, 16, 64)
    for call in (lambda: mx.quantize(x), lambda: mx.dequantize(t), lambda: mx.gemm(x, w), lambda: mx.gemm(t, w),
                 lambda: mx.tensor(t.codes, t.codes),
                 lambda: mx.grouped_gemm(x, w, torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mx.quantize([1.0]), lambda: mx.quantize(x.long()), lambda: mx.gemm(x.float(), w),
                 lambda: mx.gemm(x.numpy(), w), lambda: mx.weight(x), lambda: mx.dequantize(x)):
        with pytest.raises(TypeError):
            call()


# ---- the definitions themselves ---------------------------------------------
def test_oracle_rounds_to_even_and_saturates():
    x = torch.tensor([[4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.0, 0.26, 6.1, 7.99, -5.01, 0.0]])
    code, scale = ref.quantize(x)
    assert scale.tolist() == [[127]]
    assert ref.values(code, scale)[0].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6, 0, 0, 0.5, 6, 6, -6, 0]
    assert code[0, 9] == 8 and code[0, 10] == 8


def test_oracle_scales():
    tops = [0.0, 2.0 ** -149, 2.0 ** -126, 2.0 ** -125, 2.0 ** -124, 1.0, 1.99, 2.0, 7.99, 8.0, 2.0 ** 127, float("inf"), float("nan")]
    x = torch.zeros((len(tops), 32))
    x[:, 7] = torch.tensor(tops)
    assert ref.quantize(x)[1][:, 0].tolist() == [0, 0, 0, 0, 1, 125, 125, 126, 127, 128, 252, 255, 255]


# ---- the plans ------------------------------------------------------------------
def test_kernel_args():
    form = (ctypes.c_int32 * 4)()
    f = mx._mx().w4a16_mx_kernel
    assert f(4, 1, 40, 64, 0, 0, form) == w4.OK and f(4, 3, 40, 64, 1, 1, form) == w4.OK
    assert f(4, 1, 40, 64, 0, 0, None) == w4.ERR_NULL
    for bad in ((0, 1, 40, 64), (1 << 31, 1, 40, 64), (4, 2, 40, 64), (4, 1, 0, 64), (4, 1, 40, 60)):
        assert f(*bad, 0, 0, form) == w4.ERR_SHAPE


def form(R, N, K, quantized, experts=None):
    """A form by what the kernels' instances differ in: with parts of K or without."""
    k = mx.kernel(R, N, K, quantized, experts)
    return k if k[0] == "small" else (k[0], k[1], k[2] > 1)


def test_the_gpu_tests_have_a_shape_for_every_form():
    """Every form that some call of wide ranges of sizes takes is among those of the
    shapes that test_gpu_mx.py checks (and a split one has workspace)."""
    import random

    import test_gpu_mx as t
    rng = random.Random(0)

    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    have = {q: ({form(*s, q) for s in plain}, {form(*s[:3], q, s[3]) for s in grouped})
            for q, plain, grouped in ((False, t.FORMS16, t.GROUPED16), (True, t.FORMS4, t.GROUPED4))}
    for _ in range(6000):
        q = rng.random() < 0.5
        R, N, K = spread(1, 8192), spread(1, 32000), 8 * spread(1, 1400)
        assert form(R, N, K, q) in have[q][0], (R, N, K, q)
        assert (mx.gemm_workspace_size(R, N, K, q) > 0) == (mx.kernel(R, N, K, q)[2] > 1 and mx.kernel(R, N, K, q)[0] == "large")
        R, N, K, E = spread(1, 30000), spread(1, 8000), 8 * spread(1, 800), spread(1, 256)
        assert form(R, N, K, q, E) in have[q][1], (R, N, K, E, q)
