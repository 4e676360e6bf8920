"""The routed operators without a GPU: every symbol their header declares
resolves, and every refusal is a status of the pure-host checks."""
import ctypes
import os
import re

import pytest
import torch

import weight_only_int4_02_amd as w4
from weight_only_int4_02_amd import lora, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w4a16_routed.h")
A = 1 << 40


def P(off=0):
    return A + off


def test_every_declared_symbol_resolves():
    names = set(re.findall(r"^int32_t\s+(w4a16_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(moe.EXPORTS) | set(lora.EXPORTS)
    h = ctypes.CDLL(w4.LIB_PATH)
    for n in names:
        assert ctypes.cast(getattr(h, n), ctypes.c_void_p).value


def route(**kw):
    a = dict(logits=P(), dtype=2, T=4, E=64, bias=None, k=4, groups=1, topk=1, top=1, scale=1.0,
             flags=0, ids=P(0x1000), weights=P(0x2000))
    a.update(kw)
    return moe._routed().w4a16_check_route_args(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(), w4.OK), (dict(bias=P(4)), w4.OK), (dict(E=1024, k=32), w4.OK), (dict(k=64, E=64), w4.ERR_SHAPE),
    (dict(logits=None), w4.ERR_NULL), (dict(ids=None), w4.ERR_NULL), (dict(weights=None), w4.ERR_NULL),
    (dict(T=0), w4.ERR_SHAPE), (dict(T=(1 << 24) + 1), w4.ERR_SHAPE), (dict(E=1025), w4.ERR_SHAPE),
    (dict(E=0), w4.ERR_SHAPE), (dict(k=0), w4.ERR_SHAPE), (dict(E=3, k=4), w4.ERR_SHAPE),
    (dict(dtype=3), w4.ERR_SHAPE), (dict(dtype=-1), w4.ERR_SHAPE),
    (dict(groups=8, topk=2), w4.OK), (dict(groups=7, topk=2), w4.ERR_SHAPE),
    (dict(groups=8, topk=9), w4.ERR_SHAPE), (dict(groups=8, topk=0), w4.ERR_SHAPE),
    (dict(groups=64, topk=3, k=4), w4.ERR_SHAPE),      # three experts left for four slots
    (dict(groups=128, topk=4, E=1024), w4.ERR_SHAPE), (dict(top=3), w4.ERR_SHAPE),
    (dict(top=0), w4.ERR_SHAPE), (dict(scale=float("inf")), w4.ERR_SHAPE),
    (dict(scale=float("nan")), w4.ERR_SHAPE), (dict(flags=4), w4.ERR_FLAGS),
    (dict(logits=P(2)), w4.ERR_ALIGN), (dict(logits=P(2), dtype=0), w4.OK),
    (dict(bias=P(2)), w4.ERR_ALIGN), (dict(ids=P(2)), w4.ERR_ALIGN), (dict(weights=P(1)), w4.ERR_ALIGN),
])
def test_route_args(kw, status):
    assert route(**kw) == status


def experts(**kw):
    a = dict(X=P(), T=4, K=512, ids=P(1 << 30), weights=P(1 << 31), k=2, E=8, gq=P(), gs=P(), gz=P(),
             I=256, dq=P(), ds=P(), dz=P(), D=512, g=128, flags=0, Y=P(1 << 32), ws=P(1 << 34),
             wsb=1 << 40)
    a.update(kw)
    return moe._routed().w4a16_check_experts_args(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(), w4.OK), (dict(flags=w4.SYMMETRIC, gz=None, dz=None), w4.OK),
    (dict(X=None), w4.ERR_NULL), (dict(ids=None), w4.ERR_NULL), (dict(weights=None), w4.ERR_NULL),
    (dict(gq=None), w4.ERR_NULL), (dict(gs=None), w4.ERR_NULL), (dict(gz=None), w4.ERR_NULL),
    (dict(dz=None), w4.ERR_NULL), (dict(Y=None), w4.ERR_NULL), (dict(ws=None), w4.ERR_NULL),
    (dict(T=0), w4.ERR_SHAPE), (dict(T=1 << 21), w4.ERR_SHAPE), (dict(k=0), w4.ERR_SHAPE),
    (dict(k=33), w4.ERR_SHAPE), (dict(E=0), w4.ERR_SHAPE), (dict(E=1025), w4.ERR_SHAPE),
    (dict(T=1 << 20, k=8, K=64), w4.ERR_SHAPE),            # T k > 2^22
    (dict(K=500), w4.ERR_SHAPE), (dict(I=252), w4.ERR_SHAPE), (dict(D=0), w4.ERR_SHAPE),
    (dict(K=520), w4.ERR_GROUP), (dict(K=520, flags=w4.PARTIAL_LAST_GROUP), w4.OK),
    (dict(I=264), w4.ERR_GROUP), (dict(g=48), w4.ERR_GROUP),
    (dict(T=1 << 18, K=4096), w4.ERR_SHAPE),               # X of 2 GiB
    (dict(I=1 << 17, K=1 << 15, T=1), w4.ERR_SHAPE),       # an expert of 2^33 elements
    (dict(flags=w4.PATH_SMALL_M), w4.ERR_FLAGS), (dict(flags=0x100), w4.ERR_FLAGS),
    (dict(X=P(8)), w4.ERR_ALIGN), (dict(gq=P(4)), w4.ERR_ALIGN), (dict(dz=P(4)), w4.ERR_ALIGN),
    (dict(Y=P((1 << 32) + 2)), w4.ERR_ALIGN), (dict(ws=P(8)), w4.ERR_ALIGN),
    (dict(ids=P((1 << 30) + 2)), w4.ERR_ALIGN), (dict(ids=P((1 << 30) + 4)), w4.OK),
    (dict(wsb=16), w4.ERR_WORKSPACE), (dict(Y=P()), w4.ERR_SHAPE), (dict(ids=P(1 << 32)), w4.ERR_SHAPE),
])
def test_experts_args(kw, status):
    assert experts(**kw) == status


def test_experts_workspace_is_what_the_check_asks_for():
    for T, k, E in ((1, 1, 1), (16, 4, 8), (17, 4, 8), (1000, 8, 64)):
        b = ctypes.c_size_t()
        assert moe._routed().w4a16_experts_workspace_size(T, k, 512, 256, 512, E, 128, 0, ctypes.byref(b)) == w4.OK
        assert experts(T=T, k=k, E=E, wsb=b.value) == w4.OK
        assert experts(T=T, k=k, E=E, wsb=b.value - 1) == w4.ERR_WORKSPACE
    assert moe._routed().w4a16_experts_workspace_size(1, 1, 512, 256, 512, 1, 128, 0, None) == w4.ERR_NULL


def gemm_lora(sizes=(256, 256), **kw):
    a = dict(X=P(), M=4, K=512, q=P(), s=P(), z=P(), N=512, g=128, flags=0, A=P(), B=P(), scales=P(),
             n=4, r=16, parts=2, sizes=None, ids=P(1 << 30), Y=P(1 << 31), ws=P(1 << 34), wsb=1 << 40)
    a.update(kw)
    if sizes is not None:
        a["sizes"] = (ctypes.c_int64 * len(sizes))(*sizes)
    return lora._routed().w4a16_check_gemm_lora_args(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(), w4.OK), (dict(sizes=(512,), parts=1), w4.OK), (dict(sizes=(1, 511)), w4.OK),
    (dict(sizes=(256, 255)), w4.ERR_SHAPE), (dict(sizes=(512, 0)), w4.ERR_SHAPE),
    (dict(sizes=(600, -88)), w4.ERR_SHAPE), (dict(sizes=None), w4.ERR_NULL),
    (dict(parts=0), w4.ERR_SHAPE), (dict(parts=9), w4.ERR_SHAPE), (dict(r=12), w4.ERR_SHAPE),
    (dict(r=0), w4.ERR_SHAPE), (dict(r=264), w4.ERR_SHAPE), (dict(r=256), w4.OK), (dict(n=0), w4.ERR_SHAPE),
    (dict(n=65537), w4.ERR_SHAPE), (dict(A=None), w4.ERR_NULL), (dict(B=None), w4.ERR_NULL),
    (dict(scales=None), w4.ERR_NULL), (dict(ids=None), w4.ERR_NULL), (dict(ws=None), w4.ERR_NULL),
    (dict(X=None), w4.ERR_NULL), (dict(z=None), w4.ERR_NULL), (dict(M=0), w4.ERR_SHAPE),
    (dict(K=500), w4.ERR_SHAPE), (dict(g=100), w4.ERR_GROUP), (dict(A=P(8)), w4.ERR_ALIGN),
    (dict(B=P(2)), w4.ERR_ALIGN), (dict(scales=P(2)), w4.ERR_ALIGN), (dict(ids=P(1)), w4.ERR_ALIGN),
    (dict(ws=P(4)), w4.ERR_ALIGN), (dict(wsb=16), w4.ERR_WORKSPACE),
    (dict(Y=P()), w4.ERR_SHAPE), (dict(ids=P(1 << 31)), w4.ERR_SHAPE), (dict(flags=0x400), w4.ERR_FLAGS),
])
def test_gemm_lora_args(kw, status):
    assert gemm_lora(**kw) == status


def test_gemm_lora_workspace_is_what_the_check_asks_for():
    for M, r in ((1, 8), (4, 16), (33, 40), (700, 256)):
        b = ctypes.c_size_t()
        assert lora._routed().w4a16_gemm_lora_workspace_size(M, 512, 512, 128, 0, 2, r, ctypes.byref(b)) == w4.OK
        assert b.value >= w4.workspace_size(M, 512, 512, 128, 0) + M * 2 * r * 4
        assert gemm_lora(M=M, r=r, wsb=b.value) == w4.OK
        assert gemm_lora(M=M, r=r, wsb=b.value - 1) == w4.ERR_WORKSPACE
    assert lora._routed().w4a16_gemm_lora_workspace_size(1, 512, 512, 128, 0, 2, 16, None) == w4.ERR_NULL


def test_binding_refuses_what_it_cannot_take():
    f = torch.float32
    with pytest.raises(ValueError):
        moe.route(torch.zeros((2, 8)), 2)                       # host tensor
    with pytest.raises(TypeError):
        moe.route(torch.zeros((2, 8), dtype=torch.float64), 2)
    with pytest.raises(ValueError):
        moe.expert_weight(torch.zeros((2, 8, 32), dtype=torch.uint8), torch.zeros((2, 8, 1), dtype=torch.float16), None, 32)
    with pytest.raises(TypeError):
        lora.adapters(torch.zeros((2, 8, 32)), torch.zeros((2, 8, 8)), torch.zeros(2, dtype=f))


def test_a_layers_rows_and_logits_belong_together():
    """Shapes that only hold as many elements are refused before any call: rows
    would meet other rows' logits or adapters."""
    from weight_only_int4_02_amd.qlinear import QLinear

    def weight(N, K, gated):
        return moe.ExpertWeight(torch.zeros(0), torch.zeros(0), None, 4, N, K, 32, w4.SYMMETRIC, gated)

    layer = moe.QExperts(weight(32, 64, True), weight(64, 32, False), k=2)
    for x, logits in (((4, 64), (2, 8)), ((2, 128), (4, 4)), ((2, 3, 64), (3, 2, 4)), ((2, 3, 64), (6, 4)), ((6, 64), (24,))):
        with pytest.raises(ValueError, match="logits"):
            layer(torch.zeros(x, dtype=torch.float16), torch.zeros(logits))
    q = QLinear.__new__(QLinear)
    torch.nn.Module.__init__(q)
    q.K, q.N, q.bias, q.packed = 64, 32, None, None
    for x, ids in (((2, 3, 64), (3, 2)), ((2, 3, 64), (1, 6)), ((2, 3, 64), (2, 4)), ((6, 64), (5,))):
        with pytest.raises(ValueError, match="ids"):
            q(torch.zeros(x, dtype=torch.float16), adapters=object(), ids=torch.zeros(ids, dtype=torch.int32))
