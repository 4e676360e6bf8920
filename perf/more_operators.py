"""The measured cases of the microscaled 4-bit operators (MXFP4: blocks of 32
columns, E2M1 elements, an E8M0 scale a block): quantization, the product of
activations with such weights, and products grouped by expert over rows that
lie sorted by expert.  Activations are 16-bit, or quantized to MXFP4 in the
call ("mx").

`own` False runs each operator in its plain form (elementary torch operations
in 32 bits); `own` True makes the calls a user makes of the framework.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _quantize(name, M, K, dtype):
    case = {"op": "quantize", "M": M, "K": K, "dtype": dtype}
    return dict(case, name=name) if name else case


def _gemm(name, M, N, K, dtype, mx=False):
    case = {"op": "gemm", "M": M, "N": N, "K": K, "dtype": dtype, "mx": mx}
    return dict(case, name=name) if name else case


def _grouped(name, T, E, k, N, K, dtype, mx=False, gather=True):
    case = {"op": "grouped", "T": T, "E": E, "k": k, "N": N, "K": K, "dtype": dtype, "mx": mx,
            "gather": gather}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token's activations: the call's latency
        _quantize("quantize 1x4096 f16", 1, 4096, "f16"),
        # a ragged batch in 32 bits whose rows end inside a block
        _quantize("quantize 317x11000 f32", 317, 11000, "f32"),
        # the 7B model's gate|up weight
        _quantize("quantize 22016x4096 bf16", 22016, 4096, "bf16"),
        # one request's token through the 7B output projection
        _gemm("gemm M1 o_proj", 1, 4096, 4096, "f16"),
        # a decode batch through the fused q|k|v
        _gemm("gemm M32 qkv bf16", 32, 12288, 4096, "bf16"),
        # an odd decode batch through gate|up, activations quantized too
        _gemm("gemm M61 gate_up mx", 61, 22016, 4096, "f16", mx=True),
        # a prefill through down
        _gemm("gemm M2048 down bf16", 2048, 4096, 11008, "bf16"),
        # a prefill through gate|up, activations quantized too
        _gemm("gemm M2048 gate_up mx bf16", 2048, 22016, 4096, "bf16", mx=True),
        # one token's two of eight experts of the 7B MLP's size, gate|up
        _grouped("grouped T1 E8 7B", 1, 8, 2, 22016, 4096, "f16"),
        # a decode batch over many small experts, most touched once or twice;
        # the second product: rows in the experts' order already
        _grouped("grouped T16 E64 down bf16", 16, 64, 6, 2048, 1408, "bf16", gather=False),
        # a prefill over many small experts, activations quantized too
        _grouped("grouped T4096 E64 mx bf16", 4096, 64, 6, 2816, 2048, "bf16", mx=True),
        # a prefill through eight experts of the 7B MLP's size
        _grouped("grouped T2048 E8 7B bf16", 2048, 8, 2, 22016, 4096, "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 4e12, w["flops"] / 1e15)


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "grouped", "grouped"])
    if op == "quantize":
        M, K = _spread(rng, 1, 22016), 8 * _spread(rng, 1, 1376)
        while M > 1 and M * K > 22016 * 4096:
            M //= 2
        return _quantize(None, M, K, rng.choice(["f16", "bf16", "f32"]))
    dtype, mx = rng.choice(["f16", "bf16"]), rng.random() < 0.5
    if op == "gemm":
        M, N, K = _spread(rng, 1, 2048), _spread(rng, 64, 22016), 8 * _spread(rng, 32, 1376)
        top = _cost(listed()[7])
        while M > 1 and _cost(_gemm(None, M, N, K, dtype)) > top:
            M //= 2
        return _gemm(None, M, N, K, dtype, mx)
    E = _spread(rng, 2, 128)
    k = rng.randint(1, min(8, E))
    N, K, T = _spread(rng, 64, 4096), 8 * _spread(rng, 32, 512), _spread(rng, 1, 4096)
    top = _cost(listed()[11])
    while T > 1 and _cost(_grouped(None, T, E, k, N, K, dtype)) > top:
        T //= 2
    return _grouped(None, T, E, k, N, K, dtype, mx, rng.random() < 0.7)


def _blocks(K):
    return -(-K // BLOCK)


def _weight_bytes(N, K):
    return N * (K / 2 + _blocks(K))


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "quantize":   # values in, codes and scales out; those in, values out
        return {"bytes": int(c["M"] * (2 * c["K"] * size + 2 * (c["K"] / 2 + _blocks(c["K"])))),
                "flops": 4 * c["M"] * c["K"]}
    if c["op"] == "gemm":
        return {"bytes": int(_weight_bytes(c["N"], c["K"]) + c["M"] * (c["K"] + c["N"]) * 2),
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    R = c["T"] * c["k"]
    # experts that at least one of the rows reaches, as expected of even routing
    hit = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])
    rows = c["T"] if c["gather"] else R
    return {"bytes": int(hit * _weight_bytes(c["N"], c["K"]) + rows * c["K"] * 2 + R * c["N"] * 2 +
                         (R * 4 if c["gather"] else 0) + (c["E"] + 1) * 4),
            "flops": 2 * R * c["N"] * c["K"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _values(gen, *shape):
    """Activations: normal, a few channels an order of magnitude larger."""
    x = torch.randn(shape, device="cuda", generator=gen)
    wide = torch.rand(shape[-1], device="cuda", generator=gen) < 0.01
    return x.mul_(torch.where(wide, 8.0, 1.0))


def _weight(gen, *shape):
    """An MXFP4 weight as a checkpoint holds it: codes of a normal weight's
    sizes, two a byte (the first in the low half), and a scale byte a block."""
    K = shape[-1]
    # the codes that a block of normal values divided by its scale mostly has
    p = torch.tensor([0.13, 0.17, 0.16, 0.14, 0.17, 0.13, 0.07, 0.03], device="cuda")
    edges = p.cumsum(0)[:-1].contiguous()
    pairs = torch.rand((2, *shape[:-1], K // 2), device="cuda", generator=gen)
    code = torch.bucketize(pairs, edges, out_int32=True).to(torch.uint8)
    sign = torch.randint(0, 2, code.shape, dtype=torch.uint8, device="cuda", generator=gen)
    code = code + 8 * sign
    codes = code[0] + 16 * code[1]
    # scales around 1 / (2 sqrt(K)): outputs of unit size
    low = 127 - int(round(math.log2(2 * math.sqrt(K)))) - 1
    scales = torch.randint(low, low + 3, (*shape[:-1], _blocks(K)), dtype=torch.uint8, device="cuda",
                           generator=gen)
    return codes, scales


def _inputs(case, seed):
    """What the operator is given, before any layout of the framework's."""
    c, gen = case, _generator(seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "quantize":
        return {"X": _values(gen, c["M"], c["K"]).to(dt)}
    if c["op"] == "gemm":
        return {"X": _values(gen, c["M"], c["K"]).to(dt), "W": _weight(gen, c["N"], c["K"])}
    T, E, k = c["T"], c["E"], c["k"]
    # experts of uneven popularity, as a router gives them
    like = torch.randn((T, E), device="cuda", generator=gen) + \
        0.5 * torch.randn(E, device="cuda", generator=gen)
    ids = like.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    ends = torch.bincount(ids, minlength=E).cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    rows = (order // k).to(torch.int32) if c["gather"] else None
    return {"X": _values(gen, T if c["gather"] else T * k, c["K"]).to(dt), "W": _weight(gen, E, c["N"], c["K"]),
            "offsets": offsets, "rows": rows}


def prepare(case, seed):
    x = _inputs(case, seed)
    x["case"] = case
    if own and "W" in x:
        # the weights in the framework's layout, laid out once
        from weight_only_int4_02_amd import mx
        x["W"] = mx.weight(mx.tensor(*x["W"], case["K"]))
    return x


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _decode(codes, scales, K):
    """Code bytes [.., K/2] and scale bytes [.., blocks] -> values, in 32 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    s = torch.exp2(scales.float() - 127)
    return v * s.repeat_interleave(BLOCK, -1)[..., :K]


def _fake_quantize(x):
    """x in 32 bits -> the values of its MXFP4 form, in 32 bits."""
    K = x.shape[-1]
    v = torch.nn.functional.pad(x, (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    # frexp: a = m 2^e with m in [1/2, 1), so floor(log2 a) = e - 1
    a = v.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a).exponent - 3, -126)
    v = torch.ldexp(v, -e)
    size = v.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    v = (torch.round(v / step) * step).clamp(-6, 6)
    return torch.ldexp(v, e).flatten(-2)[..., :K]


def _plain(x):
    c = x["case"]
    X = x["X"].float()
    if c["op"] == "quantize":
        return _fake_quantize(X).to(x["X"].dtype)
    if c["mx"]:
        X = _fake_quantize(X)
    W = _decode(*x["W"], c["K"])
    if c["op"] == "gemm":
        return (X @ W.T).to(x["X"].dtype)
    if x["rows"] is not None:
        X = X[x["rows"]]
    ends = x["offsets"].tolist()
    y = torch.empty((X.shape[0], c["N"]), device=X.device)
    for e in range(c["E"]):
        if ends[e + 1] > ends[e]:
            y[ends[e]:ends[e + 1]] = X[ends[e]:ends[e + 1]] @ W[e].T
    return y.to(x["X"].dtype)


def run(state):
    x, c = state, state["case"]
    if own:
        from weight_only_int4_02_amd import mx
        if c["op"] == "quantize":
            return mx.dequantize(mx.quantize(x["X"]))
        X = mx.quantize(x["X"]) if c["mx"] else x["X"]
        if c["op"] == "gemm":
            return mx.gemm(X, x["W"])
        return mx.grouped_gemm(X, x["W"], x["offsets"], rows=x["rows"])
    return _plain(x)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_weight(codes, scales, K):
    byte = codes.to(torch.int16)
    W = torch.empty((*codes.shape[:-1], K), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        code = (byte >> (4 * half)) & 15
        mantissa, exponent = (code & 1).double(), (code >> 1) & 3
        size = torch.where(exponent == 0, 0.5 * mantissa,
                           (1 + 0.5 * mantissa) * (1 << (exponent - 1).clamp(min=0)).double())
        W[..., half::2] = torch.where(code >= 8, -size, size)
    block = torch.arange(K, device=codes.device) // BLOCK
    return W.mul_((2.0 ** (scales.double() - 127))[..., block])


def _exact_quantize(x):
    """The nearest of the eight sizes, of two the one with the even code, by
    the borders between them; a block's scale by the powers of two below its
    largest value."""
    K, x = x.shape[-1], x.double()
    out = torch.empty_like(x)
    full = K - K % BLOCK
    for part in (slice(0, full), slice(full, K)):
        v = x[:, part]
        if not v.numel():
            continue
        v = v.reshape(x.shape[0], -1, min(BLOCK, v.shape[1]))
        a = v.abs().amax(2, keepdim=True).clamp(min=2.0 ** -126)
        e = torch.floor(torch.log2(a))
        e = torch.where(2.0 ** e > a, e - 1, e)
        e = torch.where(2.0 ** (e + 1) <= a, e + 1, e)
        s = 2.0 ** (e - 2)
        size = (v / s).abs()
        level = torch.zeros_like(size)
        for border, even, up in ((0.25, True, 0.5), (0.75, False, 0.5), (1.25, True, 0.5), (1.75, False, 0.5),
                                 (2.5, True, 1.0), (3.5, False, 1.0), (5.0, True, 2.0)):
            level += up * ((size > border) if even else (size >= border))
        out[:, part] = (torch.sign(v) * level * s).reshape(x.shape[0], -1)
    return out


def exact(case, seed):
    c = case
    x = _inputs(c, seed)
    if c["op"] == "quantize":
        return _exact_quantize(x["X"])
    X = _exact_quantize(x["X"]) if c["mx"] else x["X"].double()
    if c["op"] == "gemm":
        return X @ _exact_weight(*x["W"], c["K"]).T
    y = torch.empty((c["T"] * c["k"], c["N"]), dtype=torch.float64, device=X.device)
    for e in range(c["E"]):
        at = slice(int(x["offsets"][e]), int(x["offsets"][e + 1]))
        part = X[at] if x["rows"] is None else X[x["rows"][at].long()]
        y[at] = part @ _exact_weight(x["W"][0][e], x["W"][1][e], c["K"]).T
    return y
