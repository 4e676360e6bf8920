"""Every kernel form that the plans of the routed operators can choose, on the
GPU against the definitions in 64 bits.  The cases are listed by the form they
are there for; test_forms.py checks without a GPU that none is left out."""
import pytest
import torch

import weight_only_int4_02_amd as w4
from test_gpu_lora import close, draw as draw_lora, run, weight
from test_gpu_moe import check_experts, draw as draw_experts

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

LORA_CASES = [
    # M, N, K, n, r, sizes, g.  One to four rows with the activations in LDS
    (1, 40, 1160, 3, 16, [40], 32), (1, 40, 1160, 2, 40, [24, 16], 64), (1, 40, 28008, 2, 8, [40], 32),
    (2, 16390, 1160, 2, 16, [16000, 390], 32), (2, 16390, 1160, 2, 24, [16390], 64),
    (2, 16390, 1160, 2, 64, [8195, 8195], 128),
    # weights streamed through registers, few rows
    (2, 40, 1160, 2, 48, [17, 23], 32), (1, 4200, 28680, 1, 16, [4200], 32), (2, 4200, 16392, 2, 8, [4200], 64),
    (2, 4200, 16392, 2, 64, [100, 4100], 128), (2, 4200, 1160, 2, 16, [4200], 128),
    (4, 16390, 12296, 3, 16, [16390], 128), (5, 16390, 1160, 4, 16, [5000, 11390], 32),
    (5, 16390, 1160, 4, 40, [16390], 64), (9, 40, 4200, 6, 16, [40], 32), (9, 40, 4200, 9, 64, [13, 27], 64),
    (9, 40, 4200, 5, 8, [40], 128), (17, 40, 1160, 5, 32, [40], 64), (17, 4200, 1160, 7, 16, [2100, 2100], 32),
    (17, 4200, 1160, 7, 64, [4200], 64), (17, 4200, 1160, 17, 16, [1400, 1400, 1400], 128),
    (17, 16390, 1160, 5, 16, [16390], 128), (17, 33000, 1160, 3, 40, [11000, 22000], 128),
    (33, 40, 1160, 6, 16, [40], 64),
    # activation stages through LDS
    (5, 10240, 1160, 5, 16, [10240], 128), (17, 40, 1160, 4, 24, [8, 32], 128), (17, 10240, 1160, 6, 64, [10240], 128),
    (17, 12288, 1160, 9, 16, [4096, 4096, 4096], 128), (33, 4000, 1160, 8, 16, [4000], 128),
    (33, 12288, 1160, 4, 40, [12288], 128), (33, 16390, 1160, 5, 64, [390, 16000], 128),
    (130, 4000, 648, 7, 16, [4000], 128),
    # the compute-bound tiles
    (130, 40, 648, 5, 24, [40], 32), (400, 40, 648, 4, 16, [16, 24], 128), (4096, 40, 648, 6, 16, [40], 32),
    (4096, 40, 648, 5, 48, [11, 29], 64), (130, 16390, 648, 4, 16, [16390], 32), (130, 16390, 648, 6, 64, [8000, 8390], 64),
    (65, 57344, 648, 3, 16, [57344], 128), (130, 4200, 2056, 9, 24, [2100, 2100], 128),
    (257, 22016, 648, 4, 16, [11008, 11008], 128), (528, 20480, 648, 5, 40, [20480], 128),
    (768, 16390, 648, 6, 16, [390, 8000, 8000], 128),
]

EXPERT_CASES = [
    # T, E, k, K, I, D, g.  Up to 64 slots, four weight tiles to a workgroup
    (16, 8, 3, 520, 1408, 1400, 32), (16, 8, 3, 392, 1400, 1408, 64), (16, 8, 3, 264, 1408, 2056, 128),
    # and 64-row tiles of few experts
    (50, 2, 1, 520, 264, 257, 64), (50, 2, 1, 648, 392, 130, 128),
    # planned 16-row tiles, two and four weight tiles to a workgroup
    (40, 8, 2, 392, 136, 130, 32), (40, 8, 2, 520, 264, 100, 64), (40, 64, 4, 264, 1000, 1100, 32),
    (40, 64, 4, 136, 1104, 1000, 64), (40, 64, 4, 264, 1008, 1001, 256),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,n,r,sizes,g", LORA_CASES)
def test_gemm_lora_forms(M, N, K, n, r, sizes, g, dt):
    """Rows with and without an adapter, the ones without with gemm's bits."""
    c = draw_lora(M, N, K, n, r, sizes, g, dt, symmetric=M % 2 == 0, seed=M + K,
                  ids="runs" if M > 512 else "mixed")
    if M > 2:
        c["ids"][M // 2] = -1
    if M < 3:
        c["ids"][0] = n - 1
    y = run(c)
    close(y, c)
    none = (c["ids"] < 0).cuda()
    assert torch.equal(y[none], w4.gemm(c["X"].cuda(), weight(c))[none])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,E,k,K,I,D,g", EXPERT_CASES)
def test_experts_forms(T, E, k, K, I, D, g, dt):
    for symmetric, empty in ((False, 0.0), (True, 0.2)):
        check_experts(draw_experts(T, E, k, K, I, D, g, dt, symmetric, seed=T + I, empty=empty), g)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,n,r,sizes,g,rows_each", [
    (290, 100, 264, 300, 72, [40, 1, 59], 64, 1), (520, 264, 136, 45, 64, [100, 164], 64, 2),
    (300, 700, 520, 40, 8, [700], 128, 3), (1000, 90, 64, 37, 136, [30, 33, 27], 32, 5),
    (270, 8700, 128, 60, 16, [8700], 64, 1), (200, 5000, 72, 200, 256, [2500, 2500], 256, 1)])
def test_many_adapters_in_many_rows(M, N, K, n, r, sizes, g, rows_each, dt):
    """Short runs of rows with one adapter each, in any order, some with none,
    through the compute-bound tiles: up to 128 distinct adapters in a wave's rows."""
    c = draw_lora(M, N, K, n, r, sizes, g, dt, seed=M)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(M))
    c["ids"] = order[torch.arange(M) // rows_each % n].to(torch.int32)
    c["ids"][torch.arange(0, M, 11)] = -1
    y = run(c, path="large_m")
    close(y, c)
    assert torch.equal(run(c, path="large_m"), y)
    none = (c["ids"] < 0).cuda()
    assert torch.equal(y[none], w4.gemm(c["X"].cuda(), weight(c), path="large_m")[none])
    # a broken adapter stays with its rows
    bad = int(c["ids"][1])
    c["B"][bad, 3:] = float("nan")
    rows = c["ids"] != bad
    got = run(c, path="large_m")
    assert torch.equal(got[rows.cuda()], y[rows.cuda()])
    assert bool(got[~rows.cuda(), 3:].isnan().all())
