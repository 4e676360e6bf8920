"""The measured cases of the operators in which every row of a batch meets
weights of its own: routing to experts, the experts' products over int4
weights, and low-rank adapters beside a shared int4 projection.

`own` False runs each operator in its plain form (elementary torch operations
in 32 bits, 64 where a choice lies next to a border); `own` True makes the
calls a user makes of the framework.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _route(name, T, E, k, **kw):
    case = {"op": "route", "T": T, "E": E, "k": k, "score": "softmax", "bias": False, "groups": 1,
            "topk_groups": 1, "group_top": 1, "renormalize": True, "scale": 1.0, "dtype": "f32"}
    case.update(kw)
    return dict(case, name=name) if name else case


def _experts(name, T, E, k, K, I, D, **kw):
    case = {"op": "experts", "T": T, "E": E, "k": k, "K": K, "I": I, "D": D, "g": 128,
            "symmetric": False, "empty": 0.0, "dtype": "f16"}
    case.update(kw)
    return dict(case, name=name) if name else case


def _lora(name, M, K, N, parts, n, r, **kw):
    case = {"op": "lora", "M": M, "K": K, "N": N, "parts": parts, "n": n, "r": r, "run": 1, "g": 128,
            "symmetric": False, "empty": 0.0, "dtype": "f16"}
    case.update(kw)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token of one request, a few large experts: the call's latency
        _route("route T1 E8", 1, 8, 2, dtype="f16"),
        # a decode batch of odd size over many small experts in groups; bf16
        # logits tie often
        _route("route T61 E160 groups", 61, 160, 6, dtype="bf16", groups=8, topk_groups=3,
               renormalize=False, scale=16.0),
        # a prefill's tokens, sigmoid scores with a balance bias, groups by
        # their two best
        _route("route T8192 E256 sigmoid", 8192, 256, 8, score="sigmoid", bias=True, groups=8,
               topk_groups=4, group_top=2, scale=2.5),
        # one token through two of eight experts of the 7B MLP's size
        _experts("experts T1 E8 7B", 1, 8, 2, 4096, 11008, 4096),
        # a decode batch over many small experts, most of them touched once or twice
        _experts("experts T16 E64", 16, 64, 6, 2048, 1408, 2048),
        # an odd batch in bf16, groups of 64, symmetric codes, some slots without an expert
        _experts("experts T173 E16 bf16 g64", 173, 16, 4, 2048, 1408, 2048, dtype="bf16", g=64,
                 symmetric=True, empty=0.1),
        # a prefill over many small experts in bf16, some 380 rows an expert
        _experts("experts T4096 E64 bf16", 4096, 64, 6, 2048, 1408, 2048, dtype="bf16"),
        # a prefill through eight experts of the 7B MLP's size
        _experts("experts T2048 E8 7B", 2048, 8, 2, 4096, 11008, 4096),
        # one request's token through the 7B output projection with its adapter
        _lora("lora M1 o_proj r16", 1, 4096, 4096, 1, 4, 16),
        # 32 requests, 16 adapters, through the fused q|k|v; a few without one
        _lora("lora M32 qkv r16", 32, 4096, 12288, 3, 16, 16, empty=0.1),
        # a large decode batch in bf16 through gate|up, an adapter of rank 64 for each row
        _lora("lora M61 gate_up r64 bf16", 61, 4096, 22016, 2, 61, 64, dtype="bf16"),
        # a prefill of six prompts (runs of rows with one adapter) through down
        _lora("lora M2048 down r32", 2048, 11008, 4096, 1, 6, 32, run=341),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 4e12, w["flops"] / 5e14)


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "lora", "lora"])
    dtype = rng.choice(["f16", "bf16"])
    g = rng.choice([32, 64, 128, 128, 128, 256])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _spread(rng, 4, 512 // groups)   # experts in a group
        keep = rng.randint(1, groups)
        return _route(None, _spread(rng, 1, 8192), groups * size, rng.randint(1, min(8, keep * size)),
                      dtype=rng.choice(["f16", "bf16", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                      bias=rng.random() < 0.5, groups=groups, topk_groups=keep,
                      group_top=rng.choice([1, 2]), renormalize=rng.random() < 0.7,
                      scale=rng.choice([1.0, 2.5]))
    if op == "experts":
        E = _spread(rng, 2, 128)
        k = rng.randint(1, min(8, E))
        K, I = 8 * _spread(rng, 32, 512), 8 * _spread(rng, 16, 512)
        D = K if rng.random() < 0.7 else _spread(rng, 64, 4096)
        T = _spread(rng, 1, 4096)
        top = _cost(listed()[7])
        while T > 1 and _cost(_experts(None, T, E, k, K, I, D)) > top:
            T //= 2
        return _experts(None, T, E, k, K, I, D, g=g, dtype=dtype, symmetric=rng.random() < 0.3,
                        empty=rng.choice([0.0, 0.0, 0.2]))
    parts = rng.choice([1, 1, 2, 3])
    K, N = 8 * _spread(rng, 32, 1376), parts * _spread(rng, 64, 5504)
    n = _spread(rng, 1, 64)
    M = _spread(rng, 1, 2048)
    top = _cost(listed()[11])
    r = rng.choice([8, 16, 32, 64])
    while M > 1 and _cost(_lora(None, M, K, N, parts, n, r)) > top:
        M //= 2
    return _lora(None, M, K, N, parts, n, r, run=_spread(rng, 1, max(1, M // 2)), g=g, dtype=dtype,
                 symmetric=rng.random() < 0.3, empty=rng.choice([0.0, 0.0, 0.2]))


def _weight_bytes(N, K, g, symmetric):
    G = -(-K // g)
    return N * K / 2 + N * G * 2 + (0 if symmetric else N * G / 2)


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["T"] * (c["E"] * size + c["k"] * 8), "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "experts":
        rows = c["T"] * c["k"] * (1 - c["empty"])
        # experts that at least one of the rows reaches, as expected of even routing
        hit = c["E"] * (1 - (1 - 1 / c["E"]) ** rows) if c["k"] == 1 else \
            c["E"] * (1 - (1 - c["k"] / c["E"]) ** (c["T"] * (1 - c["empty"])))
        w = _weight_bytes(2 * c["I"], c["K"], c["g"], c["symmetric"]) + \
            _weight_bytes(c["D"], c["I"], c["g"], c["symmetric"])
        return {"bytes": int(hit * w + c["T"] * (c["K"] + c["D"]) * 2 + c["T"] * c["k"] * 8),
                "flops": int(2 * rows * (2 * c["I"] * c["K"] + c["I"] * c["D"]))}
    rows = c["M"] * (1 - c["empty"])
    runs = max(1.0, rows / c["run"])
    # adapters that at least one row has
    hit = rows if c["run"] == 1 and c["n"] >= c["M"] else c["n"] * (1 - (1 - 1 / c["n"]) ** runs)
    ad = c["r"] * (c["parts"] * c["K"] + c["N"])
    return {"bytes": int(_weight_bytes(c["N"], c["K"], c["g"], c["symmetric"]) + hit * ad * 2 +
                         c["M"] * (c["K"] + c["N"]) * 2 + c["M"] * 4),
            "flops": int(2 * c["M"] * c["N"] * c["K"] + 2 * rows * ad)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _weight(gen, lead, N, K, c):
    """Codes and zeros uniform 0..15, scales that give outputs of unit size."""
    G = -(-K // c["g"])
    codes = torch.randint(0, 16, (*lead, N, K), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.rand((*lead, N, G), device="cuda", generator=gen).add_(0.5)
    scales = scales.mul_(1 / (6.5 * math.sqrt(K))).to(DTYPES[c["dtype"]])
    zeros = None if c["symmetric"] else torch.randint(0, 16, (*lead, N, G), dtype=torch.uint8,
                                                      device="cuda", generator=gen)
    return codes, scales, zeros


def _inputs(case, seed):
    """What the operator is given, before any layout of the framework's."""
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(shape, device="cuda", generator=gen)

    dt = DTYPES[c["dtype"]]
    if c["op"] == "route":
        return {"logits": normal(c["T"], c["E"]).mul_(1.5).to(dt),
                "bias": normal(c["E"]).mul_(0.05) if c["bias"] else None}
    if c["op"] == "experts":
        # experts of uneven popularity, as a router gives them
        like = normal(c["T"], c["E"]) + 0.5 * normal(c["E"])
        top = like.topk(c["k"], dim=1)
        ids = top.indices.to(torch.int32)
        ids = torch.where(uniform(c["T"], c["k"]) < c["empty"], -1, ids).to(torch.int32)
        return {"X": normal(c["T"], c["K"]).to(dt), "ids": ids, "weights": top.values.softmax(1),
                "gate_up": _weight(gen, (c["E"],), 2 * c["I"], c["K"], c),
                "down": _weight(gen, (c["E"],), c["D"], c["I"], c)}
    M, runs = c["M"], -(-c["M"] // c["run"])
    ids = torch.randint(0, c["n"], (runs,), device="cuda", generator=gen)
    if c["run"] == 1 and c["n"] >= M:      # every row an adapter of its own
        ids = torch.randperm(c["n"], device="cuda", generator=gen)[:M]
    ids = torch.where(uniform(ids.shape[0]) < c["empty"], -1, ids)
    ids = ids.repeat_interleave(c["run"])[:M].to(torch.int32).contiguous()
    return {"X": normal(M, c["K"]).to(dt), "ids": ids, "W": _weight(gen, (), c["N"], c["K"], c),
            "A": normal(c["n"], c["parts"], c["r"], c["K"]).mul_(1 / math.sqrt(c["K"])).to(dt),
            "B": normal(c["n"], c["N"], c["r"]).mul_(1 / math.sqrt(c["r"])).to(dt),
            "scales": uniform(c["n"]) + 0.5}


def prepare(case, seed):
    c = case
    x = _inputs(c, seed)
    x["case"] = c
    if own:
        # the weights and adapters in the framework's layouts, laid out once
        if c["op"] == "experts":
            from weight_only_int4_02_amd import moe
            x["gate_up"] = moe.expert_weight(*x["gate_up"], g=c["g"], gated=True)
            x["down"] = moe.expert_weight(*x["down"], g=c["g"])
        if c["op"] == "lora":
            import weight_only_int4_02_amd as w4
            from weight_only_int4_02_amd import lora
            x["W"] = w4.quantized_weight(*x["W"], c["g"], partial=c["K"] % c["g"] != 0)
            x["adapters"] = lora.adapters(x.pop("A"), x.pop("B"), x.pop("scales"),
                                          sizes=[c["N"] // c["parts"]] * c["parts"])
    return x


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _dequant(codes, scales, zeros, g):
    """W = (q - z) s rounded to the 16-bit type, in 32 bits."""
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(g, -1)[..., :codes.shape[-1]]
    s = scales.float().repeat_interleave(g, -1)[..., :codes.shape[-1]]
    return ((codes.float() - z) * s).to(scales.dtype).float()


def _plain_route(x):
    c = x["case"]
    logits = x["logits"].double()         # which score is larger is decided in 64 bits
    s = torch.softmax(logits, 1) if c["score"] == "softmax" else 1 / (1 + torch.exp(-logits))
    key = s if x["bias"] is None else s + x["bias"].double()
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        grouped = key.reshape(-1, c["groups"], size)
        value = grouped.sort(dim=2, descending=True).values[:, :, :min(c["group_top"], size)].sum(2)
        best = value.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        key = grouped.masked_fill(~keep.unsqueeze(2), -math.inf).reshape(-1, c["E"])
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = s.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _plain_experts(x):
    c = x["case"]
    ids = x["ids"].reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids + 1, minlength=c["E"] + 1).tolist()
    token, weight = order // c["k"], x["weights"].reshape(-1)[order]
    X = x["X"].float()
    y = torch.zeros((c["T"], c["D"]), device=X.device)
    at = counts[0]
    for e in range(c["E"]):
        n = counts[e + 1]
        if n:
            rows = token[at:at + n]
            gu = X[rows] @ _dequant(*[t if t is None else t[e] for t in x["gate_up"]], c["g"]).T
            gate, up = gu[:, :c["I"]], gu[:, c["I"]:]
            h = gate / (1 + torch.exp(-gate)) * up
            out = h @ _dequant(*[t if t is None else t[e] for t in x["down"]], c["g"]).T
            y.index_add_(0, rows, out * weight[at:at + n, None])
            at += n
    return y.to(x["X"].dtype)


def _plain_lora(x):
    c = x["case"]
    X = x["X"].float()
    y = X @ _dequant(*x["W"], c["g"]).T
    # every adapter's product, those of other rows' adapters set to zero
    on = x["ids"][:, None] == torch.arange(c["n"], device=X.device)
    u = (X @ x["A"].float().reshape(-1, c["K"]).T).reshape(c["M"], c["n"], c["parts"], c["r"])
    u = u * (on * x["scales"])[:, :, None, None]
    B = x["B"].float().reshape(c["n"], c["parts"], -1, c["r"])
    low = torch.matmul(u.permute(2, 0, 1, 3).reshape(c["parts"], c["M"], -1),
                       B.permute(1, 0, 3, 2).reshape(c["parts"], c["n"] * c["r"], -1).contiguous())
    return (y + low.permute(1, 0, 2).reshape(c["M"], c["N"])).to(x["X"].dtype)


def run(state):
    x, c = state, state["case"]
    if own:
        from weight_only_int4_02_amd import lora, moe
        if c["op"] == "route":
            return moe.route(x["logits"], c["k"], score=c["score"], bias=x["bias"], groups=c["groups"],
                             topk_groups=c["topk_groups"], group_top=c["group_top"],
                             renormalize=c["renormalize"], scale=c["scale"])
        if c["op"] == "experts":
            return moe.experts(x["X"], x["ids"], x["weights"], x["gate_up"], x["down"])
        return lora.gemm_lora(x["X"], x["W"], x["adapters"], x["ids"])
    return {"route": _plain_route, "experts": _plain_experts, "lora": _plain_lora}[c["op"]](x)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_weight(codes, scales, zeros, g):
    N, K = codes.shape
    W = torch.empty((N, K), dtype=torch.float64, device=codes.device)
    for j in range(scales.shape[1]):
        part = slice(j * g, min(K, (j + 1) * g))
        z = 8 if zeros is None else zeros[:, j:j + 1].long()
        W[:, part] = (codes[:, part].long() - z).double() * scales[:, j:j + 1].double()
    return W.to(scales.dtype).double()    # the exact product, rounded once


def exact(case, seed):
    c = case
    x = _inputs(c, seed)
    if c["op"] == "route":
        l = x["logits"].double()
        if c["score"] == "softmax":
            s = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        else:
            s = torch.special.expit(l)
        left = s.clone() if x["bias"] is None else s + x["bias"].double()
        rows = torch.arange(c["T"], device=l.device)
        of = torch.arange(c["E"], device=l.device) // (c["E"] // c["groups"])
        value = torch.stack([left[:, of == q].topk(min(c["group_top"], c["E"] // c["groups"]), 1).values.sum(1)
                             for q in range(c["groups"])], 1)
        for _ in range(c["groups"] - c["topk_groups"]):
            # the worst group leaves; of equal ones the last
            worst = c["groups"] - 1 - value.flip(1).argmin(1)
            value[rows, worst] = math.inf
            left[of[None, :] == worst[:, None]] = -math.inf
        w = []
        for _ in range(c["k"]):
            # the first of the largest
            at = (left == left.max(1, keepdim=True).values).to(torch.uint8).argmax(1)
            w.append(s[rows, at])
            left[rows, at] = -math.inf
        w = torch.stack(w, 1)
        return None, w * (c["scale"] / (w.sum(1, keepdim=True) if c["renormalize"] else 1))
    X = x["X"].double()
    if c["op"] == "experts":
        y = torch.zeros((c["T"], c["D"]), dtype=torch.float64, device=X.device)
        for e in range(c["E"]):
            share = (x["weights"].double() * (x["ids"] == e)).sum(1)
            rows = (x["ids"] == e).any(1).nonzero()[:, 0]
            if not len(rows):
                continue
            W = _exact_weight(*[t if t is None else t[e] for t in x["gate_up"]], c["g"])
            gate, up = X[rows] @ W[:c["I"]].T, X[rows] @ W[c["I"]:].T
            h = gate * torch.special.expit(gate) * up
            y[rows] += share[rows, None] * (h @ _exact_weight(*[t if t is None else t[e] for t in x["down"]], c["g"]).T)
        return y
    y = X @ _exact_weight(*x["W"], c["g"]).T
    step = c["N"] // c["parts"]
    for a in x["ids"].unique().tolist():
        if a < 0:
            continue
        rows = (x["ids"] == a).nonzero()[:, 0]
        for p in range(c["parts"]):
            low = X[rows] @ x["A"][a, p].double().T
            y[rows, p * step:(p + 1) * step] += x["scales"][a].double() * (
                low @ x["B"][a, p * step:(p + 1) * step].double().T)
    return y
