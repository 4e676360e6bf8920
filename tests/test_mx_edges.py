"""The microscaled 4-bit operators without a GPU: what their sources and host
checks hold at the ends of what the calls allow."""
import glob
import os
import re

import pytest

import weight_only_int4_02_amd as w4
from test_mx_abi import P, gemm, grouped
from weight_only_int4_02_amd import build, mx


def test_inline_assembly_that_writes_m0_says_so():
    """The compiler may keep a value of its own in M0: a block of assembly that
    writes the register has to name it among what it overwrites."""
    blocks = []
    for path in glob.glob(os.path.join(build.CSRC, "*")):
        blocks += re.findall(r"asm volatile\(.*?\);", open(path).read(), re.S)
    writes = [b for b in blocks if re.search(r"s_\w+ m0,", b)]
    assert writes
    for block in writes:
        assert re.search(r':\s*"m0"', block), block


# ---- results over weights --------------------------------------------------------
@pytest.mark.parametrize("quantized", [False, True])
def test_results_overlap_no_weight(quantized):
    E, N, K = 3, 40, 264
    xs = dict(xs=P(1 << 31)) if quantized else {}
    for call, n in ((lambda **kw: gemm(N=N, K=K, **xs, **kw), 1), (lambda **kw: grouped(N=N, K=K, E=E, **xs, **kw), E)):
        assert call() == w4.OK
        q, s = mx.weight_size(n, N, K)
        y = 4 * N * 2
        for size, at in ((q, 1 << 33), (s, 1 << 34)):
            for inside in (0, size - 16, 16 - y):
                assert call(Y=P(at + inside)) == w4.ERR_SHAPE
            for beside in (size, -y):
                assert call(Y=P(at + beside)) == w4.OK


@pytest.mark.parametrize("quantized", [False, True])
def test_the_workspace_overlaps_no_weight(quantized):
    shape = dict(M=61, N=64, K=11008, **(dict(xs=P(1 << 31)) if quantized else {}))
    need = mx.gemm_workspace_size(61, 64, 11008, quantized)
    assert need > 0 and need % 16 == 0 and gemm(**shape) == w4.OK
    for size, at in zip(mx.weight_size(1, 64, 11008), (1 << 33, 1 << 34)):
        for inside in (0, size - 16, 16 - need):
            assert gemm(**shape, ws=P(at + inside)) == w4.ERR_SHAPE
        for beside in (size, -need):
            assert gemm(**shape, ws=P(at + beside)) == w4.OK


def lay_out(**kw):
    """The call itself: of buffers that overlap it is refused before any launch."""
    a = dict(codes=P(), scales=P(1 << 31), E=2, N=40, K=264, q=P(1 << 33), s=P(1 << 34))
    a.update(kw)
    return mx._mx().w4a16_mx_weight(*a.values(), None)


def test_the_layout_in_place_is_refused():
    codes, scales = 2 * 40 * 256, 2 * 40 * 16
    q, s = mx.weight_size(2, 40, 264)
    for at, size in ((0, codes), (1 << 31, scales)):
        for inside in (0, size - 16):
            assert lay_out(q=P(at + inside)) == w4.ERR_SHAPE
            assert lay_out(s=P(at + inside)) == w4.ERR_SHAPE
        assert lay_out(q=P(at + 16 - q)) == w4.ERR_SHAPE
        assert lay_out(s=P(at + 16 - s)) == w4.ERR_SHAPE
    assert lay_out(s=P((1 << 33) + q - 16)) == w4.ERR_SHAPE
    assert lay_out(q=P((1 << 34) + s - 16)) == w4.ERR_SHAPE


# ---- the forms along a long K ------------------------------------------------------
def test_the_gpu_tests_have_a_shape_of_long_k_for_every_form():
    """Every form that some call with K of more than two slabs takes is among those
    of the shapes that test_gpu_mx_forms.py checks, in every type."""
    import random

    import test_gpu_mx_forms as t
    from test_mx_abi import form
    rng = random.Random(1)

    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    have = {q: ({form(*s, q) for s in plain}, {form(*s[:3], q, s[3]) for s in grouped})
            for q, plain, grouped in ((False, t.DEEP16, t.DEEP_GROUPED16), (True, t.DEEP4, t.DEEP_GROUPED4))}
    for shapes in (t.DEEP16, t.DEEP4, t.DEEP_GROUPED16, t.DEEP_GROUPED4):
        assert all(s[2] > 1024 and (s[2] % 512 or s[2] > 2048) for s in shapes)
    assert t.TYPES16 == ["f16", "bf16"]
    for _ in range(6000):
        q = rng.random() < 0.5
        R, N, K = spread(1, 8192), spread(1, 32000), 8 * spread(130, 1400)
        assert form(R, N, K, q) in have[q][0], (R, N, K, q)
        R, N, K, E = spread(1, 30000), spread(1, 8000), 8 * spread(130, 800), spread(1, 256)
        assert form(R, N, K, q, E) in have[q][1], (R, N, K, E, q)
    for q, N, K, tile in t.LAST_TILES:
        assert mx.kernel(sum(t.LAST_ROWS), N, K, q, len(t.LAST_ROWS))[:2] == ("large", tile)
