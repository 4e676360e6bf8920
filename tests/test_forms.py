"""The GPU tests' cases reach every kernel form that the host plans can choose
for the routed operators: the plans, compiled from the host sources, are asked
over a wide grid of sizes, and for the cases of the tests."""
import ctypes
import os
import subprocess

import pytest

import test_gpu_forms as forms
import test_gpu_lora as lora_tests
import test_gpu_moe as moe_tests
import weight_only_int4_02_amd as w4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_only_int4_02_amd", "csrc")

SHIM = """
#include <initializer_list>
#include "w4a16_routed.hpp"
using namespace w4a16;
extern "C" void gemm_plan(int64_t M, int64_t N, int64_t K, int32_t g, uint32_t flags, int32_t *o) {
    const GemmPlan p = plan_gemm(make_geom(M, N, K, g, flags), flags);
    const int32_t v[] = {p.path, p.lds, p.xl, p.waves, p.nb, p.depth, p.mtiles, p.large_shape};
    for (int i = 0; i < 8; i++) o[i] = v[i];
}
extern "C" void experts_plan(int64_t T, int32_t k, int64_t K, int64_t I, int64_t D, int64_t E, int32_t g,
                             uint32_t flags, int64_t *o) {
    const ExpertsPlan p = plan_experts(T, k, K, I, D, E, g, flags);
    const int64_t v[] = {p.one, p.direct, p.large, p.mt, p.bm, p.tiles};
    for (int i = 0; i < 6; i++) o[i] = v[i];
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plans")
    (d / "shim.cpp").write_text(SHIM)
    lib = str(d / "plans.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-fPIC", "-shared", "-include",
                    "initializer_list", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, str(d / "shim.cpp"),
                    os.path.join(CSRC, "w4a16_host.cpp"), os.path.join(CSRC, "w4a16_routed_host.cpp"), "-o", lib],
                   check=True)
    L = ctypes.CDLL(lib)
    I64, I32, U32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
    L.gemm_plan.argtypes = [I64, I64, I64, I32, U32, ctypes.POINTER(I32)]
    L.experts_plan.argtypes = [I64, I32, I64, I64, I64, I64, I32, U32, ctypes.POINTER(I64)]
    return L


def steps_of(g):
    """MFMA steps per group inside a 128-column tile: the kernels' group class."""
    return min(g // 32, 4)


def gemm_form(L, M, N, K, g, bf):
    o = (ctypes.c_int32 * 8)()
    L.gemm_plan(M, N, K, g, w4.BF16 if bf else 0, o)
    path, lds, xl, waves, nb, depth, mtiles, shape = o
    if path == 0:
        return ("small", bf, steps_of(g), "lds" if lds else "xl" if xl else "registers", waves, nb, depth,
                0 if lds else mtiles)
    if g < 128:   # (the launcher's tiles for small groups)
        shape = {12: 3, 14: 3, 17: 3, 20: 3, 21: 3, 18: 0}.get(shape, shape)
    return "large", bf, steps_of(g), shape


def expert_forms(L, T, E, k, K, I, D, g, bf, symmetric):
    o = (ctypes.c_int64 * 6)()
    L.experts_plan(T, k, K, I, D, E, g, (w4.BF16 if bf else 0) | (w4.SYMMETRIC if symmetric else 0), o)
    one, direct, large, mt, bm, tiles = o
    if one:
        return {("one", bf, steps_of(g), product) for product in ("gate_up", "down")}
    if large:
        return {("large", bf, steps_of(g), bm, product) for product in ("gate_up", "down")}
    # (the launcher takes four weight tiles to a workgroup where they are many)
    return {("small", bf, steps_of(g), "direct" if direct else "planned", mt,
             4 if mt == 1 and tiles * ((-(-N // 16) + 1) // 2) >= 2048 else 2, product)
            for product, N in (("gate_up", I), ("down", D))}


def test_every_gemm_form_has_an_adapter_case(plans):
    cases = lora_tests.CASES + forms.LORA_CASES
    have = {gemm_form(plans, M, N, K, g, bf) for M, N, K, _, _, _, g in cases for bf in (False, True)}
    Ms = list(range(1, 72)) + list(range(80, 544, 16)) + [640, 768, 1024, 1500, 2048, 4096]
    Ns = [16, 96, 256, 1000, 2048, 4096, 4112, 5120, 7168, 8192, 10240, 11008, 12288, 14336, 16384, 20480, 22016,
          28672, 33000, 57344]
    Ks = [64, 256, 512, 1024, 2048, 4096, 5120, 8192, 11008, 16384, 20480, 28672]
    reach = {}
    for bf in (False, True):
        for g in (32, 64, 128):
            for M in Ms:
                for N in Ns:
                    for K in Ks:
                        reach.setdefault(gemm_form(plans, M, N, K, g, bf), (M, N, K, g))
    assert len(reach) > 80
    assert not {f: at for f, at in reach.items() if f not in have}


def test_every_experts_form_has_a_case(plans):
    cases = moe_tests.CASES + forms.EXPERT_CASES
    have = set()
    for T, E, k, K, I, D, g in cases:
        for bf in (False, True):
            for symmetric in (False, True):
                have |= expert_forms(plans, T, E, k, K, I, D, g, bf, symmetric)
    reach = {}
    for bf in (False, True):
        for g in (32, 64, 128):
            for symmetric in (False, True):
                for T in (1, 2, 5, 16, 40, 64, 100, 173, 300, 1000, 4096):
                    for E in (1, 2, 3, 4, 8, 16, 64, 128):
                        for k in (1, 2, 4, 6, 8):
                            for K in (128, 2048, 4096):
                                for I in (128, 1408, 11008):
                                    for D in (128, 2048, 4096):
                                        for f in expert_forms(plans, T, E, k, K, I, D, g, bf, symmetric):
                                            reach.setdefault(f, (T, E, k, K, I, D, g))
    assert len(reach) > 80
    assert not {f: at for f, at in reach.items() if f not in have}
