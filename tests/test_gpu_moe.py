"""Routing and the experts' products on the GPU against their definitions in
64 bits (oracle/routed.py), whose bounds are derived there."""
import pytest
import torch

import weight_only_int4_02_amd as w4
from oracle import routed as ref
from weight_only_int4_02_amd import moe

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check_route(logits, k, **kw):
    bias = kw.pop("bias", None)
    ids, w = moe.route(logits.cuda(), k, bias=None if bias is None else bias.cuda(), **kw)
    want_ids, want, bound = ref.route(logits, k, bias=bias, **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert torch.equal(ids.cpu(), want_ids)
    off = (w.cpu().double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 64, 6), (4, 65, 8), (130, 128, 8),
                                   (33, 256, 32), (5, 511, 7), (2, 1024, 16), (2001, 160, 6),
                                   # many rows: several to a wave
                                   (2049, 8, 2), (2065, 16, 16), (2050, 31, 20), (2100, 64, 8),
                                   (2051, 100, 32), (2500, 250, 8), (2052, 256, 8), (2053, 300, 3)])
def test_route_plain(T, E, k, dt):
    l = torch.randn((T, E), generator=gen(T + E)).mul(2).to(DT[dt])
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            check_route(l, k, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,topk,k", [(8, 2, 1, 4), (64, 64, 5, 5), (160, 8, 3, 6), (256, 8, 4, 8), (60, 4, 4, 9)])
@pytest.mark.parametrize("T", [65, 2061])
def test_route_groups_and_bias(T, E, groups, topk, k, biased, group_top, score):
    l = torch.randn((T, E), generator=gen(E))
    bias = torch.randn(E, generator=gen(E + 1)).mul(0.1) if biased else None
    check_route(l, k, score=score, bias=bias, groups=groups, topk_groups=topk, group_top=group_top)


def test_route_ties_go_to_the_lowest_index():
    l = torch.randint(-2, 3, (2300, 96), generator=gen(3)).float()
    for rows in (300, 2300):
        check_route(l[:rows], 8)
    for kw in (dict(), dict(score="sigmoid"), dict(groups=8, topk_groups=3),
               dict(groups=8, topk_groups=3, group_top=2), dict(bias=torch.zeros(96))):
        check_route(l, 8, **kw)
    check_route(torch.zeros((5, 200)), 8)


def test_route_excluded_experts_and_odd_values():
    inf, nan = float("inf"), float("nan")
    l = torch.randn((12, 16), generator=gen(4))
    l[0] = -inf                       # nothing left
    l[1] = nan
    l[2, 3:] = -inf                   # three left for four slots
    l[3, 5] = inf
    l[4, :] = inf
    l[5, 2] = nan
    l[6] = 3e38
    l[7] = -3e38
    l[8, ::2] = -inf
    l[9, :8] = -inf                   # whole groups
    l[10, 1:] = -1000.0               # scores that vanish in 32 bits
    lowest = torch.finfo(torch.float32).min
    l[11, 4:] = lowest                # the type's lowest value is a value
    bias = torch.zeros(16)
    bias[1], bias[2], bias[15] = -inf, nan, -0.5
    for rows in (l, l.repeat(180, 1)):
        check_route(rows, 4)
        check_route(rows, 4, score="sigmoid")
        check_route(rows, 4, renormalize=False)
        check_route(rows, 4, groups=4, topk_groups=2)
        check_route(rows, 4, groups=4, topk_groups=2, group_top=2)
        check_route(rows, 4, score="sigmoid", bias=bias)
        check_route(rows, 4, score="sigmoid", bias=bias, groups=4, topk_groups=2, group_top=2)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T", [40, 2100])
def test_route_sigmoid_of_very_negative_logits(T, dt):
    """Scores far below what 32 bits hold still weigh against each other: whole
    rows of logits from -85 to -700 (their 64-bit scores are normal numbers),
    with and without a bias of zeros, which takes the keys' wider form."""
    E, k = 16, 4
    low = torch.linspace(-85, -700, T)[:, None]
    l = (low - torch.rand((T, E), generator=gen(5)) * 5).to(DT[dt])
    l[0, :4] = torch.tensor([-90.0, -91.0, -95.0, -100.0])
    l[0, 4:] = -float("inf")
    zeros = torch.zeros(E)
    check_route(l, k, score="sigmoid")
    check_route(l, k, score="sigmoid", renormalize=False, scale=2.5)
    # (groups judged by their best alone: the logits are the keys there too)
    check_route(l, k, score="sigmoid", groups=4, topk_groups=2)
    ids, w = moe.route(l.cuda(), k, score="sigmoid")
    assert bool(((w.sum(1) - 1).abs() < 1e-5).all())
    # a bias of zeros: the same weights wherever it leaves the same experts
    ids0, w0 = moe.route(l.cuda(), k, score="sigmoid", bias=zeros.cuda())
    assert torch.equal(ids, ids0) and torch.equal(w, w0)


def test_route_empty_and_refusals():
    ids, w = moe.route(torch.zeros((0, 8), device="cuda"), 2)
    assert tuple(ids.shape) == (0, 2) and tuple(w.shape) == (0, 2)
    x = torch.zeros((4, 8), device="cuda")
    for bad in (dict(k=9), dict(k=0), dict(k=2, groups=3), dict(k=2, score="max"),
                dict(k=2, bias=torch.zeros(7, device="cuda")), dict(k=2, groups=2, topk_groups=3),
                dict(k=2, scale=float("inf"))):
        with pytest.raises(ValueError):
            moe.route(x, **bad)
    with pytest.raises(ValueError):
        moe.route(torch.zeros((0, 8), device="cuda"), 9)
    with pytest.raises(ValueError):
        moe.route(x.t(), 2)
    with pytest.raises(TypeError):
        moe.route(x, 2, bias=torch.zeros(8, dtype=torch.float16, device="cuda"))


# ---- the experts' products --------------------------------------------------
def draw(T, E, k, K, I, D, g, dt, symmetric, seed, empty=0.0):
    r = gen(seed)

    def weight(N, Kc):
        G = -(-Kc // g)
        codes = torch.randint(0, 16, (E, N, Kc), dtype=torch.uint8, generator=r)
        scales = (torch.rand((E, N, G), generator=r) + 0.5).div(6.5 * Kc ** 0.5).to(DT[dt])
        zeros = None if symmetric else torch.randint(0, 16, (E, N, G), dtype=torch.uint8, generator=r)
        return codes, scales, zeros

    X = torch.randn((T, K), generator=r).to(DT[dt])
    ids = torch.stack([torch.randperm(E, generator=r)[:k] for _ in range(T)]).to(torch.int32)
    ids = torch.where(torch.rand((T, k), generator=r) < empty, -1, ids).to(torch.int32)
    return X, ids, torch.rand((T, k), generator=r), weight(2 * I, K), weight(D, I)


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]


def on_gpu(case, g):
    X, ids, w, gu, dn = case
    return (X.cuda(), ids.cuda(), w.cuda(), moe.expert_weight(*cuda(gu), g=g, gated=True),
            moe.expert_weight(*cuda(dn), g=g))


def check_experts(case, g, **kw):
    X, ids, w, gu, dn = case
    y = moe.experts(*on_gpu(case, g), **kw)
    want, bound = ref.experts(X, ids, w, gu, dn, g)
    off = (y.cpu().double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    return y


CASES = [
    # T, E, k, K, I, D, g: the direct form up to 64 rows, the planned one above;
    # 16-row and 64-row tiles; ragged K, I, D
    (1, 1, 1, 128, 128, 16, 128), (1, 8, 2, 256, 128, 128, 128), (2, 3, 3, 264, 136, 100, 128),
    (7, 4, 2, 512, 256, 257, 64), (16, 4, 4, 256, 384, 256, 32), (64, 2, 1, 136, 72, 17, 32),
    (33, 8, 2, 520, 200, 264, 256), (40, 2, 2, 256, 264, 256, 128), (100, 16, 4, 384, 128, 130, 128),
    (200, 3, 1, 1024, 104, 64, 64), (300, 4, 4, 256, 256, 512, 128),
    # one token: many slots, partial stages, and an activation image too large
    (1, 16, 8, 264, 200, 100, 32), (1, 4, 4, 1160, 648, 257, 64), (1, 4, 4, 128, 11008, 64, 128),
    (1, 3, 2, 4096, 1408, 2048, 256), (1, 32, 32, 128, 136, 48, 128), (1, 2, 2, 128, 14336, 32, 128),
    # the compute-bound kernel: 64-row and 128-row tiles, every group size,
    # K of one, few and many stages, ragged columns and a partial last stage
    (130, 8, 2, 128, 136, 257, 32), (150, 6, 2, 392, 512, 260, 64), (129, 4, 1, 648, 72, 300, 256),
    (333, 2, 1, 264, 640, 516, 32), (257, 3, 3, 1160, 264, 131, 64), (500, 2, 1, 512, 1032, 640, 256),
    (140, 1, 1, 128, 128, 16, 128), (700, 5, 2, 640, 200, 1100, 128),
    # more slots than workgroups, with a last round cut into half slots and
    # tiles of few rows among the whole ones
    (1500, 4, 1, 128, 8192, 264, 128), (1400, 4, 1, 256, 136, 20000, 64), (900, 3, 1, 136, 10000, 9000, 32),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,E,k,K,I,D,g", CASES)
def test_experts(T, E, k, K, I, D, g, dt):
    for symmetric, empty in ((False, 0.0), (True, 0.3)):
        check_experts(draw(T, E, k, K, I, D, g, dt, symmetric, seed=T + K, empty=empty), g)


@pytest.mark.parametrize("T", [5, 90])
def test_experts_rows_without_an_expert(T):
    """ids outside 0..E-1 add nothing, whole rows of them are 0, and an id twice
    in a row counts twice; nothing of the slots' weights is looked at."""
    case = draw(T, 4, 3, 256, 128, 128, 128, "f16", False, seed=T)
    X, ids, w = case[:3]
    ids[0] = -1
    ids[1] = torch.tensor([4, 1 << 30, -(1 << 31)])
    ids[2] = 1
    ids[3] = torch.tensor([2, -7, 2])
    w[0], w[1] = float("nan"), float("inf")
    clean = (X, ids, torch.where(torch.isfinite(w), w, torch.zeros(())), *case[3:])
    Xc, idc, wc, gu, dn = on_gpu(case, 128)
    y = moe.experts(Xc, idc, wc, gu, dn)
    want, bound = ref.experts(*clean, 128)
    assert bool(((y.cpu().double() - want).abs() <= bound).all())
    assert not y[:2].any()
    none = moe.experts(Xc, torch.full_like(idc, -1), wc, gu, dn)
    assert none.shape == y.shape and not none.any()
    assert tuple(moe.experts(Xc[:0], idc[:0], wc[:0], gu, dn).shape) == (0, 128)


@pytest.mark.parametrize("ids", [[2, 2, 0], [-1, 3, 99], [-1, 4, -5], [3, -1, 3]])
def test_one_token(ids):
    """A single row's form: an expert twice, slots without one (whose weights,
    NaN here, are not looked at), and none at all."""
    case = draw(1, 4, 3, 520, 264, 100, 128, "f16", False, seed=7)
    case[1][:] = torch.tensor(ids)
    for j, e in enumerate(ids):
        case[2][0, j] = 0.25 + j if 0 <= e < 4 else float("nan")
    X, i, w, gu, dn = on_gpu(case, 128)
    y = moe.experts(X, i, w, gu, dn)
    want, bound = ref.experts(case[0], case[1], torch.nan_to_num(case[2], 0.0), *case[3:], 128)
    assert bool(((y.cpu().double() - want).abs() <= bound).all())
    assert y.any() == any(0 <= e < 4 for e in ids)


@pytest.mark.parametrize("T,all_one", [(64, True), (300, True), (300, False)])
def test_experts_all_rows_on_one_expert(T, all_one):
    """Tiles of one expert, the others idle; and an infinity or NaN in one row
    of X stays in that row."""
    case = draw(T, 5, 1, 256, 128, 128, 128, "bf16", False, seed=T)
    if all_one:
        case[1][:] = 4
    X = case[0]
    X[3, 5], X[9, 0] = float("inf"), float("nan")
    y = moe.experts(*on_gpu(case, 128)).cpu()
    fine = torch.ones(T, dtype=torch.bool)
    fine[3] = fine[9] = False
    want, bound = ref.experts(X[fine], case[1][fine], case[2][fine], case[3], case[4], 128)
    assert bool(((y[fine].double() - want).abs() <= bound).all())
    assert not torch.isfinite(y[9]).any()


@pytest.mark.parametrize("T,E,k,K,I,D,g,symmetric", [
    (1, 4, 2, 256, 264, 100, 128, False), (1, 3, 3, 520, 136, 257, 32, True),      # one token
    (5, 4, 2, 256, 136, 130, 64, False), (50, 2, 1, 264, 200, 64, 128, True),      # direct
    (90, 8, 2, 256, 136, 257, 32, False),                                          # planned 16-row tiles
    (150, 6, 2, 392, 264, 260, 64, False), (300, 4, 2, 256, 136, 520, 128, True)]) # 64- and 128-row tiles
def test_experts_beyond_fp16_on_the_way(T, E, k, K, I, D, g, symmetric):
    """fp16: silu(gate) up far beyond 65504 that the down projection brings back
    into range, in some columns of every row, beside rows without any."""
    case = draw(T, E, k, K, I, D, g, "f16", symmetric, seed=T + I, empty=0.1 if T > 1 else 0.0)
    X, ids, w, gu, dn = case
    gu = (gu[0], (gu[1].double() * 300).half(), gu[2])
    dn = (dn[0], (dn[1].double() * 2.0 ** -7).half(), dn[2])
    X[3::4] = (X[3::4].double() / 64).half()         # rows that stay in range
    w[:, 0] = torch.where(torch.arange(T) % 3 == 0, 0.0, w[:, 0])    # a slot of no weight beside them
    h_max = (X[0].double() @ ref.weight(*[t if t is None else t[int(ids[0, -1])] for t in gu], g).T).abs().max() ** 2
    assert h_max > 2 * 65504
    y = check_experts((X, ids, w, gu, dn), g)
    assert torch.isfinite(y).all()
    # an infinity in one row of X stays in that row
    if T > 1:
        X[4, 7] = float("inf")
        ids[4] = torch.arange(k)
        y = moe.experts(*on_gpu((X, ids, w, gu, dn), g)).cpu()
        fine = torch.arange(T) != 4
        want, bound = ref.experts(X[fine], ids[fine], w[fine], gu, dn, g)
        assert bool(((y[fine].double() - want).abs() <= bound).all())
        assert not torch.isfinite(y[4]).any()


def test_experts_of_more_rows_than_one_grid_axis():
    """The weighted sum's rows over two axes of its grid, one of the last rows
    beyond fp16 on the way."""
    T, E, k, K, I, D, g = 33000, 2, 2, 64, 64, 20, 32
    X, ids, w, gu, dn = draw(T, E, k, K, I, D, g, "f16", False, seed=1, empty=0.1)
    gu = (gu[0], (gu[1].double() * 100).half(), gu[2])
    X = (X.double() / 40).half()
    X[32900] = (X[32900].double() * 80).half()
    ids[32900] = torch.tensor([1, 0])
    case = X, ids, w, gu, (dn[0], (dn[1].double() / 64).half(), dn[2])
    h = X[32900].double() @ ref.weight(*[t[1] for t in gu], g).T
    assert (torch.nn.functional.silu(h[:I]) * h[I:]).abs().max() > 65504
    y = check_experts(case, g)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("T", [1, 5, 90, 300])
def test_experts_of_rows_that_are_not_finite(T):
    """fp16: NaN and infinities in X, in routing weights and scales, without any
    h that overflows: what the definition gives, NaN where it does."""
    case = draw(T, 4, 2, 256, 136, 100, 128, "f16", False, seed=T)
    X, ids, w, gu, dn = case
    X[0, 3] = float("nan")
    y = moe.experts(*on_gpu(case, 128)).cpu()
    assert bool(y[0].isnan().all()) and bool(torch.isfinite(y[1:]).all())
    X[0, 3] = 1.0
    w[0, 0] = float("inf")
    y = moe.experts(*on_gpu(case, 128)).cpu()
    assert not torch.isfinite(y[0]).any() and bool(torch.isfinite(y[1:]).all())
    w[0, 0] = 0.5
    dn[1][:, 7] = float("inf")     # one column of every expert
    y = moe.experts(*on_gpu(case, 128)).cpu()
    assert not torch.isfinite(y[:, 7]).any()
    rest = torch.cat([y[:, :7], y[:, 8:]], 1)
    want, bound = ref.experts(X, ids, w, gu, (dn[0], torch.where(torch.isinf(dn[1]), 0.0, dn[1]).half(), dn[2]), 128)
    want, bound = [torch.cat([t[:, :7], t[:, 8:]], 1) for t in (want, bound)]
    assert bool(((rest.double() - want).abs() <= bound).all())


def test_experts_is_repeatable_and_keeps_its_neighbours():
    """The same bits each time, into a caller's output and workspace, and
    nothing written before or behind them."""
    case = draw(120, 8, 3, 256, 136, 72, 128, "f16", False, seed=8)
    args = on_gpu(case, 128)
    y = moe.experts(*args)
    T, D = y.shape
    need = moe.experts_workspace_size(T, 3, args[3], args[4])
    block = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    rows = torch.full((T + 2, D), 7.0, dtype=torch.float16, device="cuda")
    for _ in range(3):
        got = moe.experts(*args, out=rows[1:-1], workspace=block[256:256 + need])
        assert got.data_ptr() == rows[1:-1].data_ptr()
        assert torch.equal(got, y)
    assert bool((rows[0] == 7).all()) and bool((rows[-1] == 7).all())
    assert bool((block[:256] == 0x5A).all()) and bool((block[256 + need:] == 0x5A).all())
    with pytest.raises(ValueError):
        moe.experts(*args, workspace=block[:need - 256])


def test_experts_refusals():
    case = draw(4, 4, 2, 256, 128, 128, 128, "f16", False, seed=1)
    X, ids, w, gu, dn = on_gpu(case, 128)
    other = on_gpu(draw(4, 4, 2, 256, 128, 128, 128, "bf16", False, seed=1), 128)
    sym = on_gpu(draw(4, 4, 2, 256, 128, 128, 128, "f16", True, seed=1), 128)
    for bad in ((X, ids, w, dn, gu), (X, ids, w, gu, gu), (X[:, :128].contiguous(), ids, w, gu, dn),
                (X, ids[:2], w, gu, dn), (X, ids, w[:, :1].contiguous(), gu, dn), (X.t(), ids, w, gu, dn)):
        with pytest.raises(ValueError):
            moe.experts(*bad)
    for bad in ((X.float(), ids, w, gu, dn), (X, ids.long(), w, gu, dn), (X, ids, w.half(), gu, dn),
                (other[0], ids, w, gu, dn), (X, ids, w, gu, sym[4]), (X, ids, w, other[3], other[4])):
        with pytest.raises(TypeError):
            moe.experts(*bad)
    gu.q = gu.q[:-1]
    with pytest.raises(ValueError):
        moe.experts(X, ids, w, gu, dn)
    with pytest.raises(ValueError):
        moe.expert_weight(*cuda((case[3][0][:, :255], case[3][1][:, :255], case[3][2][:, :255])), g=128, gated=True)


@pytest.mark.parametrize("T,E", [(1, 8), (21, 8), (150, 16)])
def test_router_and_experts_together(T, E):
    """The layer as it is served: logits -> route -> experts, captured in a graph
    and replayed with other inputs between eager calls, on a stream of its own."""
    k, K, I, g = 3, 256, 128, 64
    case = draw(T, E, k, K, I, K, g, "bf16", False, seed=T)
    _, _, _, gu, dn = on_gpu(case, g)
    bias = torch.randn(E, generator=gen(1)).mul(0.1)
    kw = dict(score="sigmoid", bias=bias, groups=4, topk_groups=2, group_top=2, scale=2.0)
    layer = moe.QExperts(gu, dn, k, **{**kw, "bias": bias.cuda()})
    xs = [torch.randn((T, K), generator=gen(s)).to(torch.bfloat16) for s in range(3)]
    ls = [torch.randn((T, E), generator=gen(10 + s)) for s in range(3)]

    def check(y, s):
        ids, w, _ = ref.route(ls[s], k, **kw)
        want, bound = ref.experts(xs[s], ids, w, case[3], case[4], g)
        # (the weights' own rounding to 32 bits: below 2^-20 of the result's terms)
        bound = bound + 2.0 ** -20 * bound / (torch.finfo(torch.bfloat16).eps / 2)
        assert bool(((y.cpu().double() - want).abs() <= bound).all())

    side = torch.cuda.Stream()
    x, l = xs[0].cuda().reshape(1, T, K), ls[0].cuda().reshape(1, T, E)
    out = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(side):
        y = layer(x, l)
        assert y.shape == (1, T, K)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer(x, l, out=out)
    side.synchronize()
    check(y.reshape(T, K), 0)
    for s in (1, 2, 0, 1):
        x.copy_(xs[s].reshape(1, T, K))
        l.copy_(ls[s].reshape(1, T, E))
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(out, s)
        eager = layer(x, l)
        torch.cuda.synchronize()
        assert torch.equal(eager.reshape(T, K), out)


def test_calls_on_two_streams_at_once():
    """Calls without a workspace of their own, on two streams that nothing
    orders: each has its own block, eager and in two graphs replayed in turn."""
    cases = [draw(T, 8, 3, 256, 128, 256, 64, "f16", False, seed=20 + T) for T in (150, 21)]
    args = [on_gpu(c, 64) for c in cases]
    want = [moe.experts(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(8):
        got = []
        for st, a in zip(streams, args):
            with torch.cuda.stream(st):
                got.append(moe.experts(*a))
        torch.cuda.synchronize()
        for y, w in zip(got, want):
            assert torch.equal(y, w)
    graphs = []
    for st, a, o in zip(streams, args, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.stream(st), torch.cuda.graph(graphs[-1], stream=st):
            moe.experts(*a, out=o)
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for y, w, a in zip(outs, want, args):
            assert torch.equal(y, w)
            assert torch.equal(moe.experts(*a), w)
        torch.cuda.synchronize()


def test_sizes_that_are_refused_before_memory_is_taken():
    logits = torch.zeros((1 << 10, 8), device="cuda")
    for k in (0, -1, 9, 33, 1 << 40, (1 << 32) + 1):
        with pytest.raises(ValueError):
            moe.route(logits, k)
    codes = torch.zeros((2, 32, 64), dtype=torch.uint8, device="cuda")
    scales = torch.ones((2, 32, 2), dtype=torch.float16, device="cuda")
    for g in (0, -32):
        with pytest.raises(ValueError):
            moe.expert_weight(codes, scales, None, g)
    with pytest.raises(ValueError):
        moe.expert_weight(codes, scales.cpu(), None, 32)


@pytest.mark.parametrize("n,symmetric", [(40, False), (16, True), (33, True)])
def test_expert_weight_is_each_matrix_repacked(n, symmetric):
    """The matrices in the device layout, one after the other, also where their
    rows end inside a tile."""
    E, K, g = 3, 200, 64
    codes = torch.randint(0, 16, (E, 2 * n, K), generator=gen(n), dtype=torch.uint8).cuda()
    scales = torch.rand((E, 2 * n, 4), generator=gen(n + 1)).half().cuda()
    zeros = None if symmetric else torch.randint(0, 16, (E, 2 * n, 4), generator=gen(n + 2), dtype=torch.uint8).cuda()
    got = moe.expert_weight(codes, scales, zeros, g, gated=True)
    one = [w4.repack(w4.pack(codes[e, r].contiguous()), scales[e, r].clone(),
                     None if symmetric else w4.pack(zeros[e, r].contiguous()), K, g, symmetric=symmetric, partial=True)
           for e in range(E) for r in (slice(0, n), slice(n, 2 * n))]
    assert torch.equal(got.q.flatten(), torch.cat([w.q for w in one]))
    assert torch.equal(got.s.flatten(), torch.cat([w.s for w in one]))
    assert symmetric or torch.equal(got.z.flatten(), torch.cat([w.z for w in one]))


@pytest.mark.parametrize("E,groups,topk,k", [(264, 8, 3, 6), (512, 4, 2, 8), (500, 5, 2, 4), (1000, 8, 4, 8), (1024, 64, 9, 32),
                                             (1024, 2, 1, 3), (96, 32, 7, 11), (240, 15, 4, 8)])
@pytest.mark.parametrize("T", [9, 2070])
def test_route_groups_of_every_width(T, E, groups, topk, k):
    """Groups of one lane's experts, of several lanes' and of parts of a lane's;
    some rows with whole groups excluded, some with equal logits throughout."""
    l = torch.randn((T, E), generator=gen(E + groups))
    l[3, : 2 * (E // groups)] = float("-inf")
    l[5] = 1.0
    l[7, E // groups - 1 :] = float("-inf")
    bias = torch.randn(E, generator=gen(E)).mul(0.1)
    for kw in (dict(), dict(group_top=2), dict(bias=bias, score="sigmoid"), dict(bias=bias, group_top=2)):
        check_route(l, k, groups=groups, topk_groups=topk, **kw)
