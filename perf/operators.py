"""Measured cases of the operators for layers with experts and 4-bit weights: routing tokens to
experts, quantising to microscaled 4-bit floats (MX FP4: blocks of 32 values along the contracted
axis, each value e2m1, one power-of-two scale per block), the product of two such operands, and
the products of every expert with the rows routed to it.

With `own` false, `run` computes an operator in its plain form, from elementary torch operations;
with `own` true it makes the calls of concurrent_gemm_dma_amd that a user's program makes.

Layout of an MX FP4 operand of `rows` x `cols`: codes [rows][P/2] (low nibble = even column) and
scales [rows][P/32] (exponent + 127), where P is cols rounded up to 256 and what is past cols is
zero. Slots: the j-th choice of token t is slot j*T + t.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of e2m1 by code
LARGEST = float(np.finfo(np.float32).max)

# ---- cases --------------------------------------------------------------------------------------


def listed():
    return [
        # one token's activations of a 16384-wide model before a 4-bit product: latency
        {"name": "quantise one token", "op": "quantise", "rows": 1, "cols": 16384, "dtype": "bf16",
         "transpose": False, "rule": "floor"},
        # a prefill or training batch of activations, row by row
        {"name": "quantise 8192 tokens", "op": "quantise", "rows": 8192, "cols": 16384,
         "dtype": "bf16", "transpose": False, "rule": "floor"},
        # the gradient of a 28672-wide up-projection, blocks along the tokens: the operand of the
        # weight gradient in training
        {"name": "quantise gradient, transposed", "op": "quantise", "rows": 8192, "cols": 28672,
         "dtype": "bf16", "transpose": True, "rule": "up"},
        # a single token through a 70B-class up-projection: decoding, bound by the weights' bytes
        {"name": "product, one token", "op": "product", "M": 1, "N": 28672, "K": 8192,
         "out": "bf16"},
        # a ragged batch, no size a multiple of a tile
        {"name": "product, ragged batch", "op": "product", "M": 777, "N": 4999, "K": 4000,
         "out": "bf16"},
        # the 405B-class up-projection of a full batch
        {"name": "product, 405B-class", "op": "product", "M": 8192, "N": 53248, "K": 16384,
         "out": "bf16"},
        # eight decoding sequences over 32 experts: one or two rows an expert
        {"name": "experts, decode", "op": "experts", "T": 8, "E": 32, "k": 4, "N": 4096, "K": 4096,
         "skew": 0.5, "masked": 0.0, "out": "bf16"},
        # ragged sizes, uneven load, some experts without rows, some tokens without experts
        {"name": "experts, ragged and skewed", "op": "experts", "T": 1001, "E": 24, "k": 3,
         "N": 2072, "K": 2720, "skew": 2.0, "masked": 0.1, "out": "bf16"},
        # a prefill batch over 8 experts, two each
        {"name": "experts, prefill", "op": "experts", "T": 8192, "E": 8, "k": 2, "N": 14336,
         "K": 4096, "skew": 0.5, "masked": 0.0, "out": "bf16"},
        # one decoding token, sigmoid scores, balance bias, the best 4 of 8 groups by their top two
        {"name": "route, one token", "op": "route", "T": 1, "E": 256, "k": 8, "score": "sigmoid",
         "groups": 8, "top_groups": 4, "group_top": 2, "bias": True, "renorm": True,
         "dtype": "f32", "masked": 0.0},
        # a long prefill, softmax over 128 experts, bf16 logits with ties
        {"name": "route, 32768 tokens", "op": "route", "T": 32768, "E": 128, "k": 8,
         "score": "softmax", "groups": 1, "top_groups": 1, "group_top": 1, "bias": False,
         "renorm": True, "dtype": "bf16", "masked": 0.0},
        # a training batch: the logits' gradient from the weights' gradient
        {"name": "route backward, 8192 tokens", "op": "route_backward", "T": 8192, "E": 256,
         "k": 8, "score": "sigmoid", "groups": 8, "top_groups": 4, "group_top": 2, "bias": True,
         "renorm": True, "dtype": "bf16", "masked": 0.01},
    ]


def draw(rng):
    def size(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    op = rng.choice(("quantise", "product", "experts", "route", "route_backward"))
    if op == "quantise":
        rows = size(1, 8192)
        return {"op": op, "rows": rows, "cols": size(32, 28672), "dtype": rng.choice(("bf16", "f32")),
                "transpose": rng.random() < 0.4, "rule": rng.choice(("floor", "up"))}
    if op == "product":
        return {"op": op, "M": size(1, 8192), "N": size(64, 53248), "K": size(64, 16384),
                "out": rng.choice(("bf16", "bf16", "f32"))}
    if op == "experts":
        E, K = size(4, 64), size(256, 8192)
        N = size(256, min(8192, 470_000_000 // (E * K)))  # no more weights than a listed case has
        return {"op": op, "T": size(1, 8192), "E": E, "k": rng.randint(1, 4), "N": N, "K": K, "skew": round(rng.uniform(0.0, 2.0), 2), "masked": rng.choice((0.0, 0.1)), "out": rng.choice(("bf16", "bf16", "f32"))}
    groups = rng.choice((1, 1, 4, 8))
    E = groups * size(4, 256 // groups)
    k = rng.randint(1, min(8, E // groups))
    return {"op": op, "T": size(1, 32768), "E": E, "k": k, "score": rng.choice(("softmax", "sigmoid")),
            "groups": groups, "top_groups": rng.randint(1, groups), "group_top": rng.choice((1, 2)),
            "bias": rng.random() < 0.5, "renorm": rng.random() < 0.6,
            "dtype": rng.choice(("bf16", "f32")), "masked": rng.choice((0.0, 0.05))}


def work(case):
    op = case["op"]
    if op == "quantise":
        n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        # x read; codes, scales and the values that they stand for written
        return {"bytes": n * (size + 17 / 32 + 2), "flops": 2 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * 17 / 32 + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    if op == "experts":
        slots, N, K = case["T"] * case["k"], case["N"], case["K"]
        size = 2 if case["out"] == "bf16" else 4
        # of the experts' weights those that some slot can reach
        return {"bytes": (case["T"] + min(case["E"], slots) * N) * K * 17 / 32 + slots * N * size
                + 8 * slots, "flops": 2 * slots * N * K}
    T, E, k, size = case["T"], case["E"], case["k"], 2 if case["dtype"] == "bf16" else 4
    if op == "route":  # logits read; indices, weights, order and offsets written
        return {"bytes": T * E * size + T * k * 12 + 4 * (E + 1), "flops": 4 * T * E}
    # logits, indices and the weights' gradient read; the logits' gradient written
    return {"bytes": 2 * T * E * size + T * k * 8, "flops": 4 * T * E}


# ---- inputs -------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _padded(cols):
    return (cols + 255) // 256 * 256


def _quantise(x, rule="floor"):
    """Codes (one a byte) and scale bytes of fp32 x [..., cols], cols a multiple of 32."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)  # amax = m * 2^e with 0.5 <= m < 1
    # floor(log2 amax) - 2 = e - 3; the block then reaches below 8, and 6 is the largest code
    e = e - 3 if rule == "floor" else e - 3 + (m > 0.75).to(e.dtype)
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(min=-127))
    # the factor 2^-e in two halves: 2^127 * 2^-... stays a normal number
    y = torch.ldexp(torch.ldexp(b, -(e // 2)), -(e - e // 2))
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8) + 8 * torch.signbit(y).to(torch.uint8))
    fine = torch.isfinite(amax)
    code = torch.where(fine, code, torch.zeros_like(code))
    scale = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return code.reshape(x.shape), scale.squeeze(-1)


def _operand(x):
    """An MX FP4 operand of x [..., cols]: packed codes and scales."""
    cols = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, _padded(cols) - cols))
    code, scale = _quantise(x)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), scale.contiguous()


def _logits(case, g):
    T, E = case["T"], case["E"]
    x = 1.5 * torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    if case["masked"]:  # experts out of reach, some tokens without any
        x.masked_fill_(torch.rand(T, E, generator=g, device=DEV) < case["masked"], -math.inf)
        x.masked_fill_(torch.rand(T, 1, generator=g, device=DEV) < 0.2 * case["masked"], -math.inf)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
    return x.to(_dtype(case["dtype"])), bias


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    if op == "quantise":
        rows, cols = case["rows"], case["cols"]
        x = torch.randn(rows, cols, generator=g, device=DEV)
        if case["rule"] == "up":  # gradients: small, and of uneven size from row to row
            x *= 1e-4 * torch.exp(torch.randn(rows, 1, generator=g, device=DEV))
        r, c = (cols, rows) if case["transpose"] else (rows, cols)
        empty = lambda *shape: torch.empty(*shape, dtype=torch.uint8, device=DEV)  # noqa: E731
        return {"case": case, "x": x.to(_dtype(case["dtype"])), "codes": empty(r, _padded(c) // 2),
                "scales": empty(r, _padded(c) // 32),
                "values": torch.empty(r, c, dtype=torch.bfloat16, device=DEV)}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        a, sa = _operand(torch.randn(M, K, generator=g, device=DEV))
        b, sb = _operand(0.02 * torch.randn(N, K, generator=g, device=DEV))
        return {"case": case, "a": a, "sa": sa, "b": b, "sb": sb,
                "C": torch.empty(M, N, dtype=_dtype(case["out"]), device=DEV)}
    if op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        a, sa = _operand(torch.randn(T, K, generator=g, device=DEV))
        b, sb = _operand(0.02 * torch.randn(E, N, K, generator=g, device=DEV))
        # the k experts of every token, uneven over the experts; masked: tokens without experts
        z = torch.randn(T, E, generator=g, device=DEV) + case["skew"] * torch.randn(E, generator=g, device=DEV)
        idx = z.topk(k, dim=1).indices.to(torch.int32)
        if case["masked"]:
            idx.masked_fill_(torch.rand(T, 1, generator=g, device=DEV) < case["masked"], -1)
        weights = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1).contiguous()
        order, offsets = _plan(idx, E)
        return {"case": case, "a": a, "sa": sa, "b": b, "sb": sb, "weights": weights,
                "order": order, "offsets": offsets,
                "most": int((offsets[1:] - offsets[:-1]).max()),  # rows of the busiest expert
                "C": torch.empty(T * k, N, dtype=_dtype(case["out"]), device=DEV)}
    x, bias = _logits(case, g)
    T, E, k = case["T"], case["E"], case["k"]
    s = {"case": case, "logits": x, "bias": bias}
    if op == "route":
        whole = lambda *shape: torch.empty(*shape, dtype=torch.int32, device=DEV)  # noqa: E731
        s |= {"idx": whole(T, k), "weights": torch.empty(T, k, device=DEV), "order": whole(T * k),
              "offsets": whole(E + 1)}
    else:
        s |= {"idx": _choose(x, bias, case).to(torch.int32).contiguous(),
              "dweights": torch.randn(T, k, generator=g, device=DEV), "dlogits": torch.empty_like(x)}
    return s


# ---- plain forms --------------------------------------------------------------------------------


def _values(codes, scales, cols):
    """fp32 values [..., cols] of packed codes and scale bytes."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), device=DEV)
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    s = torch.where(scales == 255, math.nan, torch.ldexp(torch.ones_like(scales, dtype=torch.float32),
                                                         scales.to(torch.int32) - 127))
    v = table[code.long()].reshape(*scales.shape, 32) * s.unsqueeze(-1)
    return v.flatten(-2)[..., :cols]


def _scores(x, case):
    """(reachable, logits, scores) in 64 bits: choices between near scores need them."""
    reach = x > -math.inf  # false for NaN too
    l = x.double().clamp(max=LARGEST)
    if case["score"] == "sigmoid":
        s = torch.where(l >= 0, 1 / (1 + torch.exp(-l.abs())), torch.exp(-l.abs()) / (1 + torch.exp(-l.abs())))
    else:
        top = l.masked_fill(~reach, -LARGEST).amax(1, keepdim=True)
        s = torch.exp((l - top).masked_fill(~reach, -math.inf))
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    return reach, l, s.masked_fill(~reach, 0.0)


def _choose(x, bias, case):
    """Indices [T][k] of the chosen experts, best first, -1 where there is none."""
    reach, l, s = _scores(x, case)
    b = 0.0 if bias is None else bias.double()
    v = (l if bias is None else s + b).masked_fill(~reach, -math.inf)
    G = case["groups"]
    if G > 1:
        by = v.reshape(v.shape[0], G, -1)
        if case["group_top"] == 2:  # the two best by v, their scores with the bias added up
            two = by.sort(dim=2, descending=True, stable=True).indices[..., :2]
            w = (s + b).masked_fill(~reach, 0.0).reshape(by.shape).gather(2, two).sum(2)
            of = w.masked_fill(~(by > -math.inf).any(2), -math.inf)
        else:
            of = by.amax(2)
        best = of.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros_like(of, dtype=torch.bool).scatter_(1, best, True)
        v = by.masked_fill(~keep.unsqueeze(2), -math.inf).flatten(1)
    v, idx = v.sort(dim=1, descending=True, stable=True)
    return idx[:, :case["k"]].masked_fill(~(v[:, :case["k"]] > -math.inf), -1)


def _plan(idx, E):
    """(order, offsets): the slots j*T + t by expert, within an expert by token; absent last."""
    T, k = idx.shape
    e = torch.where((idx >= 0) & (idx < E), idx, E).reshape(-1)
    at = e.sort(stable=True).indices
    order = (at % k * T + at // k).to(torch.int32)
    offsets = torch.searchsorted(e.sort().values, torch.arange(E + 1, device=DEV, dtype=e.dtype))
    return order, offsets.to(torch.int32)


def _route(s):
    case, x, bias = s["case"], s["logits"], s["bias"]
    idx = _choose(x, bias, case)
    absent, at = idx < 0, idx.clamp(min=0)
    l = x.double().clamp(max=LARGEST).gather(1, at)
    if case["renorm"]:  # the chosen scores over their sum, scaled by a power of e that cancels
        top = l.masked_fill(absent, -LARGEST).amax(1, keepdim=True)
        if case["score"] == "sigmoid":
            top = top.clamp(max=0.0)
            w = torch.where(l > 0, 1 / (1 + torch.exp(-l)), torch.exp(l - top) / (1 + torch.exp(l)))
        else:
            w = torch.exp(l - top)
        w = w.masked_fill(absent, 0.0)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = _scores(x, case)[2].gather(1, at).masked_fill(absent, 0.0)
    idx = idx.to(torch.int32)
    order, offsets = _plan(idx, case["E"])
    return {"idx": idx, "weights": w.float(), "order": order, "offsets": offsets}


def _route_backward(s):
    case, x = s["case"], s["logits"]
    absent, at = s["idx"] < 0, s["idx"].clamp(min=0).long()
    g = s["dweights"].masked_fill(absent, 0.0)
    reach = x > -math.inf
    l = x.float().clamp(max=LARGEST)
    if case["score"] == "sigmoid":
        p, q = torch.sigmoid(l.gather(1, at)), torch.sigmoid(-l.gather(1, at))
        p = p.masked_fill(absent, 0.0)
        if case["renorm"]:
            w = p / p.sum(1, keepdim=True).clamp(min=1e-37)
            d = q * w * (g - (g * w).sum(1, keepdim=True))
        else:
            d = g * p * q
        return torch.zeros_like(l).scatter_add_(1, at, d.masked_fill(absent, 0.0)).to(x.dtype)
    top = l.masked_fill(~reach, -LARGEST).amax(1, keepdim=True)
    p = torch.exp((l - top).masked_fill(~reach, -math.inf))
    if case["renorm"]:  # a softmax over the chosen
        c = l.gather(1, at)
        w = torch.exp((c - c.masked_fill(absent, -LARGEST).amax(1, keepdim=True)).masked_fill(absent, -math.inf))
        w = w / w.sum(1, keepdim=True).clamp(min=1e-37)
        d = w * (g - (g * w).sum(1, keepdim=True))
        return torch.zeros_like(l).scatter_add_(1, at, d.masked_fill(absent, 0.0)).to(x.dtype)
    p = p / p.sum(1, keepdim=True).clamp(min=1e-37)
    inner = (g * p.gather(1, at)).sum(1, keepdim=True)
    return (p * (torch.zeros_like(l).scatter_add_(1, at, g) - inner)).to(x.dtype)


def _experts(s):
    case = s["case"]
    T, E, k, K = (case[n] for n in ("T", "E", "k", "K"))
    order, offsets = s["order"].long(), s["offsets"].long()
    i = torch.arange(T * k, device=DEV)
    e = (torch.searchsorted(offsets, i, right=True) - 1).clamp(max=E - 1)
    absent = i >= offsets[E]
    rank = (i - offsets[e]).masked_fill(absent, s["most"])  # row `most` of each pad is not used
    t, j = order % T, order // T
    pad = torch.zeros(E, s["most"] + 1, K, device=DEV)
    pad[e, rank] = _values(s["a"], s["sa"], K)[t]
    y = torch.matmul(pad, _values(s["b"], s["sb"], K).transpose(1, 2).contiguous())
    y = y[e, rank] * s["weights"][t, j].masked_fill(absent, 0.0).unsqueeze(1)
    return torch.empty_like(y).index_copy_(0, order, y.masked_fill(absent.unsqueeze(1), 0.0)).to(_dtype(case["out"]))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantise":
        x = (s["x"].t() if case["transpose"] else s["x"]).float()
        cols = x.shape[1]
        code, scale = _quantise(torch.nn.functional.pad(x, (0, _padded(cols) - cols)), case["rule"])
        return _values(code[:, 0::2] | (code[:, 1::2] << 4), scale, cols).to(torch.bfloat16)
    if op == "product":
        A, B = _values(s["a"], s["sa"], case["K"]), _values(s["b"], s["sb"], case["K"])
        return torch.matmul(A, B.t()).to(_dtype(case["out"]))
    return {"experts": _experts, "route": _route, "route_backward": _route_backward}[op](s)


# ---- the framework's operators ------------------------------------------------------------------

_lib = None


def _framework():
    global _lib
    if _lib is None:
        from concurrent_gemm_dma_amd import _c3

        _c3.c3_init(0)
        _lib = _c3
    return _lib


def _options(c3, case):
    return c3.route_opts(score=c3.C3_SCORE_SIGMOID if case["score"] == "sigmoid" else c3.C3_SCORE_SOFTMAX,
                         top_k=case["k"], n_groups=case["groups"], top_groups=case["top_groups"],
                         group_top=case["group_top"], renormalize=case["renorm"], scale=1.0)


def _calls(s):
    c3, case = _framework(), s["case"]
    op = case["op"]
    kind = lambda name: c3.C3_BF16 if name == "bf16" else c3.C3_F32  # noqa: E731
    if op == "quantise":
        rows, cols = case["rows"], case["cols"]
        c3.c3_mx4_quantize(s["x"], kind(case["dtype"]), rows, cols, cols, case["transpose"],
                           c3.C3_MX4_UP if case["rule"] == "up" else c3.C3_MX4_FLOOR, s["codes"], s["scales"])
        if case["transpose"]:
            rows, cols = cols, rows
        c3.c3_mx4_dequantize(s["codes"], s["scales"], rows, cols, s["values"], c3.C3_BF16, cols)
        return s["values"]
    if op == "product":
        c3.c3_mx4_gemm(s["a"], s["sa"], s["b"], s["sb"], s["C"], kind(case["out"]), case["M"], case["N"],
                       case["K"], case["N"])
        return s["C"]
    if op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        c3.c3_mx4_gemm_experts(s["a"], s["sa"], T, s["b"], s["sb"], s["order"], s["offsets"], s["weights"],
                               s["C"], kind(case["out"]), T, k, E, N, K, N)
        return s["C"]
    T, E, k, o = case["T"], case["E"], case["k"], _options(c3, case)
    if op == "route":
        c3.c3_route(s["logits"], kind(case["dtype"]), T, E, E, o, s["bias"], s["idx"], s["weights"])
        c3.c3_route_plan(s["idx"], T, k, E, s["order"], s["offsets"])
        return {n: s[n] for n in ("idx", "weights", "order", "offsets")}
    c3.c3_route_backward(s["logits"], kind(case["dtype"]), T, E, E, o, s["idx"], s["dweights"], s["dlogits"], E)
    return s["dlogits"]


def run(state):
    return _calls(state) if own else _plain(state)


# ---- definitions in 64 bits ---------------------------------------------------------------------


def _decoded(codes, scales, cols):
    """float64 values of an operand, from the bits of e2m1: sign, two exponent bits, one more."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2((e - 1).double()) * (1 + 0.5 * m)) * (1 - 2 * (n >> 3)).double()
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1))[..., :cols]


def _exact_quantise(s):
    case = s["case"]
    x = (s["x"].t() if case["transpose"] else s["x"]).double()
    cols = x.shape[1]
    b = torch.nn.functional.pad(x, (0, -cols % 32)).unflatten(1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True).clamp(min=1e-300)
    unit = torch.exp2(torch.floor(torch.log2(amax)) - 2)
    if case["rule"] == "up":
        unit = torch.where(amax > 6 * unit, 2 * unit, unit)
    unit = unit.clamp(min=2.0 ** -127)
    y = b / unit
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1.0))) - 1)  # distance of neighbours
    return ((y / step).round() * step).clamp(-6, 6).mul_(unit).flatten(1)[:, :cols]


def _exact_experts(s):
    case = s["case"]
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    at, order = s["offsets"].tolist(), s["order"].long()
    A = _decoded(s["a"], s["sa"], K)
    C = torch.zeros(T * k, N, dtype=torch.float64, device=DEV)
    for e in range(E):
        p = order[at[e]:at[e + 1]]
        W = _decoded(s["b"][e], s["sb"][e], K)
        C[p] = (A[p % T] @ W.t()) * s["weights"].double()[p % T, p // T].unsqueeze(1)
    return C


def _exact_weights(x, idx, case):
    """(weights of the chosen, probabilities of all) in float64, on the host."""
    l = x.double().cpu().numpy().clip(max=LARGEST)
    l[np.isnan(l)] = -np.inf
    idx = idx.cpu().numpy().astype(np.int64)
    with np.errstate(all="ignore"):
        # log of each score; what all scores of a row share cancels in the sum's quotient
        log = -np.logaddexp(0, -l) if case["score"] == "sigmoid" else l
        if case["score"] == "softmax":
            log = log - np.logaddexp.reduce(log, axis=1, keepdims=True)
        c = np.where(idx < 0, -np.inf, np.take_along_axis(log, idx.clip(min=0), 1))
        if case["renorm"]:
            c = c - np.logaddexp.reduce(c, axis=1, keepdims=True)
    return np.where(idx < 0, 0.0, np.exp(c)), np.where(np.isneginf(l), 0.0, np.exp(log)), l, idx


def _exact_route(s):
    case = s["case"]
    idx = _choose(s["logits"], s["bias"], case)
    w = _exact_weights(s["logits"], idx, case)[0]
    return {"idx": None, "weights": torch.from_numpy(w), "order": None, "offsets": None}


def _exact_route_backward(s):
    case = s["case"]
    w, p, l, idx = _exact_weights(s["logits"], s["idx"], case)
    g = np.where(idx < 0, 0.0, s["dweights"].double().cpu().numpy())
    inner = (g * w).sum(1, keepdims=True)
    d = np.zeros_like(p)
    rows, cols = np.nonzero(idx >= 0)
    at = idx[rows, cols]
    if case["score"] == "sigmoid":
        q = 1 / (1 + np.exp(l[rows, at]))
        d[rows, at] = q * (w * (g - inner if case["renorm"] else g))[rows, cols]
    elif case["renorm"]:
        d[rows, at] = (w * (g - inner))[rows, cols]
    else:
        d = -p * inner
        d[rows, at] += (w * g)[rows, cols]
    return torch.from_numpy(d)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "product":
        return _decoded(s["a"], s["sa"], case["K"]) @ _decoded(s["b"], s["sb"], case["K"]).t()
    return {"quantise": _exact_quantise, "experts": _exact_experts, "route": _exact_route,
            "route_backward": _exact_route_backward}[op](s)
