"""Measured cases of the operators that carry tokens to their experts and back, and of expert layers
in 8-bit integers: rows sorted by expert (as they are, or quantised on the way), the weighted sum
that brings them back, its gradient, and the products of int8 operands with a scale for each token
and each channel, of one matrix or of every expert's.

With `own` false, `run` computes an operator in its plain form, from elementary torch operations;
with `own` true it makes the calls of concurrent_gemm_dma_amd that a user's program makes.

Layout of an int8 operand of `rows` x `cols`: codes [rows][P] with P = cols rounded up to 128, zeros
past cols, and scales [rows] fp32. A row's scale is a / 127, a its largest magnitude; its codes are
x * r rounded to the nearest integer, ties to even, with r = 127 / a rounded to fp32. Slots: the j-th
choice of token t is slot j*T + t; pos[slot] is its row in expert order, -1 without an expert.
"""
import math

import torch

own = False

DEV = "cuda:0"
SMALLEST = 2.0 ** -119  # a row's largest magnitude counts as this at least

# ---- cases --------------------------------------------------------------------------------------


def listed():
    return [
        # one token's activations before an 8-bit product: latency
        {"name": "quantise one token", "op": "quantise", "T": 1, "E": 0, "k": 1, "cols": 16384,
         "dtype": "bf16", "sort": False, "masked": 0.0},
        # a prefill batch sent to its experts as 8-bit rows: half the bytes of the all-to-all
        {"name": "quantise and sort 8192 tokens", "op": "quantise", "T": 8192, "E": 64, "k": 4,
         "cols": 8192, "dtype": "bf16", "sort": True, "masked": 0.0},
        # a single token through a 70B-class up-projection: decoding, bound by the weights' bytes
        {"name": "int8 product, one token", "op": "product", "M": 1, "N": 28672, "K": 8192, "out": "bf16"},
        # the same projection of a full batch
        {"name": "int8 product, 8192 tokens", "op": "product", "M": 8192, "N": 28672, "K": 8192, "out": "bf16"},
        # eight decoding sequences over 32 experts: one or two rows an expert
        {"name": "int8 experts, decode", "op": "experts", "T": 8, "E": 32, "k": 4, "N": 4096, "K": 4096,
         "skew": 0.5, "masked": 0.0, "out": "bf16"},
        # an odd prefill batch over 8 experts of uneven load, two each, some tokens without any
        {"name": "int8 experts, uneven prefill", "op": "experts", "T": 8191, "E": 8, "k": 2, "N": 14336,
         "K": 4096, "skew": 1.0, "masked": 0.05, "out": "bf16"},
        # eight decoding sequences sorted by expert: latency
        {"name": "sort, decode", "op": "dispatch", "T": 8, "E": 32, "k": 4, "cols": 4096, "dtype": "bf16",
         "masked": 0.0},
        # a long prefill of eight choices each: the send buffer of the all-to-all
        {"name": "sort 32768 tokens", "op": "dispatch", "T": 32768, "E": 128, "k": 8, "cols": 4096,
         "dtype": "bf16", "masked": 0.0},
        # the way back of the decoding step
        {"name": "combine, decode", "op": "combine", "T": 8, "E": 32, "k": 4, "cols": 4096, "dtype": "bf16",
         "weighted": True, "masked": 0.0},
        # the way back of the long prefill
        {"name": "combine 32768 tokens", "op": "combine", "T": 32768, "E": 128, "k": 8, "cols": 4096,
         "dtype": "bf16", "weighted": True, "masked": 0.0},
        # a small training batch in fp32, ragged, some tokens without experts
        {"name": "combine backward, ragged", "op": "combine_backward", "T": 1001, "E": 24, "k": 3,
         "cols": 2720, "dtype": "f32", "masked": 0.1},
        # a training batch: gradients of the experts' rows and of the routing weights
        {"name": "combine backward, 8192 tokens", "op": "combine_backward", "T": 8192, "E": 256, "k": 8,
         "cols": 8192, "dtype": "bf16", "masked": 0.01},
    ]


def draw(rng):
    def size(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    op = rng.choice(("quantise", "product", "experts", "dispatch", "combine", "combine_backward"))
    if op == "product":
        return {"op": op, "M": size(1, 8192), "N": size(64, 28672), "K": size(64, 8192),
                "out": rng.choice(("bf16", "bf16", "f32"))}
    if op == "experts":
        E, K = size(4, 64), size(256, 8192)
        N = size(256, min(8192, 470_000_000 // (E * K)))  # no more weights than a listed case has
        return {"op": op, "T": size(1, 8192), "E": E, "k": rng.randint(1, 4), "N": N, "K": K,
                "skew": round(rng.uniform(0.0, 2.0), 2), "masked": rng.choice((0.0, 0.1)),
                "out": rng.choice(("bf16", "bf16", "f32"))}
    cols, dtype = size(64, 16384), rng.choice(("bf16", "bf16", "f32"))
    if rng.random() < 0.5:
        cols = max(64, cols // 64 * 64)
    k = rng.randint(1, 8)
    # elements of all slots: no more bytes than a listed case moves
    most = {"quantise": 1 << 28, "combine_backward": 1 << 29}.get(op, 1 << 30) // (2 if dtype == "f32" else 1)
    case = {"op": op, "T": size(1, min(32768, most // (k * cols))), "E": size(8, 256), "k": k, "cols": cols,
            "dtype": dtype, "masked": rng.choice((0.0, 0.05))}
    if op == "quantise":
        case["sort"] = rng.random() < 0.5
        if not case["sort"]:
            case |= {"E": 0, "k": 1, "masked": 0.0}
    if op == "combine":
        case["weighted"] = rng.random() < 0.7  # unweighted: the gradient of the sort
    return case


def work(case):
    op = case["op"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K + 4) + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    if op == "experts":
        slots, N, K = round(case["T"] * case["k"] * (1 - case["masked"])), case["N"], case["K"]
        # of the experts' weights those that some row can reach
        return {"bytes": (slots + min(case["E"], slots) * N) * (K + 4)
                + slots * N * (2 if case["out"] == "bf16" else 4) + 4 * (case["E"] + 1), "flops": 2 * slots * N * K}
    T, k, cols, size = case["T"], case["k"], case["cols"], 2 if case["dtype"] == "bf16" else 4
    slots, plan = round(T * k * (1 - case["masked"])), 8 * T * k  # slots without an expert have no row
    if op == "quantise":  # x read; codes, scales and the values that they stand for written; the plan
        return {"bytes": T * cols * size + slots * (cols * 3 + 4) + (plan if case["sort"] else 0),
                "flops": 3 * slots * cols}
    if op == "dispatch":  # x read, the sorted rows written; order read, positions written
        return {"bytes": (T + slots) * cols * size + plan, "flops": 0}
    if op == "combine":  # sorted rows, positions and weights read; the sums written
        return {"bytes": (T + slots) * cols * size + plan, "flops": 2 * slots * cols}
    # the sums' gradient, the rows, positions and weights read; the rows' and weights' gradients written
    return {"bytes": (T + 2 * slots) * cols * size + plan + 4 * slots, "flops": 3 * slots * cols}


# ---- inputs -------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _padded(cols):
    return (cols + 127) // 128 * 128


def _quantise(x):
    """(codes as float64, scales fp32) of x [rows][cols]."""
    a = x.float().abs().amax(1, keepdim=True).clamp(min=SMALLEST)
    r = 127.0 / a
    return torch.round(x.double() * r.double()), (a / 127.0).squeeze(1)  # the product is exact in 64 bits


def _operand(x):
    """An int8 operand of x [rows][cols]."""
    codes, scales = _quantise(x)
    return torch.nn.functional.pad(codes.to(torch.int8), (0, _padded(x.shape[1]) - x.shape[1])), scales


def _activations(rows, cols, g):
    """Activations: channels of uneven size, a few of them far larger than the others."""
    channel = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    channel = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.005, 20 * channel, channel)
    return torch.randn(rows, cols, generator=g, device=DEV) * channel


def _weights(experts, N, K, g):
    """An int8 operand of (experts * N) x K, made expert by expert."""
    codes = torch.zeros(experts * N, _padded(K), dtype=torch.int8, device=DEV)
    scales = torch.empty(experts * N, device=DEV)
    for e in range(experts):
        for n in range(0, N, 8192):
            rows = slice(e * N + n, e * N + min(N, n + 8192))
            x = 0.02 * torch.randn(rows.stop - rows.start, K, generator=g, device=DEV)
            codes[rows], scales[rows] = _operand(x)
    return codes, scales


def _routing(case, g):
    """(order, offsets) of the k experts of every token, uneven over the experts."""
    T, E, k = case["T"], case["E"], case["k"]
    z = torch.randn(T, E, generator=g, device=DEV)
    z += case.get("skew", 0.5) * torch.randn(E, generator=g, device=DEV)
    e = z.topk(k, dim=1).indices
    if case["masked"]:  # tokens without experts
        e = e.masked_fill(torch.rand(T, 1, generator=g, device=DEV) < case["masked"], E)
    e = e.reshape(-1)
    at = e.sort(stable=True).indices
    order = (at % k * T + at // k).to(torch.int32)
    offsets = torch.searchsorted(e.sort().values, torch.arange(E + 1, device=DEV, dtype=e.dtype))
    return order, offsets.to(torch.int32)


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": case}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["sa"] = _operand(_activations(M, K, g))
        s["b"], s["sb"] = _weights(1, N, K, g)
        return s | {"C": torch.empty(M, N, dtype=_dtype(case["out"]), device=DEV)}
    if op == "experts":
        E, N, K, slots = case["E"], case["N"], case["K"], case["T"] * case["k"]
        s["a"], s["sa"] = _operand(_activations(slots, K, g))
        s["b"], s["sb"] = _weights(E, N, K, g)
        s["offsets"] = _routing(case, g)[1]
        # rows without an expert are left as they were: zeros here
        return s | {"host": s["offsets"].tolist(), "C": torch.zeros(slots, N, dtype=_dtype(case["out"]), device=DEV)}
    T, k, cols, dtype = case["T"], case["k"], case["cols"], _dtype(case["dtype"])
    slots = T * k
    if op == "quantise":
        s["x"] = _activations(T, cols, g).to(dtype)
        if case["sort"]:
            s["order"], s["offsets"] = _routing(case, g)
            s["pos"] = torch.empty(k, T, dtype=torch.int32, device=DEV)
        return s | {"codes": torch.zeros(slots, _padded(cols), dtype=torch.int8, device=DEV),
                    "scales": torch.zeros(slots, device=DEV),
                    "values": torch.empty(slots, cols, dtype=torch.bfloat16, device=DEV)}
    s["order"], s["offsets"] = _routing(case, g)
    if op == "dispatch":
        return s | {"x": torch.randn(T, cols, generator=g, device=DEV).to(dtype),
                    "y": torch.zeros(slots, cols, dtype=dtype, device=DEV),
                    "pos": torch.empty(k, T, dtype=torch.int32, device=DEV)}
    s["pos"] = _positions(s)
    s["y"] = torch.empty(slots, cols, dtype=dtype, device=DEV)
    for row in range(0, slots, 32768):
        s["y"][row:row + 32768].normal_(generator=g)
    s["weights"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1).contiguous()
    if op == "combine":
        if not case["weighted"]:
            s["weights"] = None
        return s | {"out": torch.empty(T, cols, dtype=dtype, device=DEV)}
    return s | {"dout": torch.randn(T, cols, generator=g, device=DEV).to(dtype),
                "dy": torch.zeros(slots, cols, dtype=dtype, device=DEV),
                "dweights": torch.empty(T, k, device=DEV)}


# ---- plain forms --------------------------------------------------------------------------------


def _positions(s):
    """pos [k][T]: the row of each slot in expert order, -1 without an expert."""
    T, k = s["case"]["T"], s["case"]["k"]
    row = torch.arange(T * k, device=DEV, dtype=torch.int32)
    row = torch.where(row < s["offsets"][-1], row, -1)
    return torch.empty_like(row).scatter_(0, s["order"].long(), row).view(k, T)


def _present(s):
    """Truth values [slots][1] of the rows that belong to an expert."""
    return (torch.arange(s["order"].numel(), device=DEV) < s["offsets"][-1]).unsqueeze(1)


def _sorted(s, x):
    return torch.where(_present(s), x[s["order"].long() % s["case"]["T"]], torch.zeros((), dtype=x.dtype, device=DEV))


def _product(a, b):
    """float64 sums a . b^T of codes. 1024 products of codes are exact in fp32."""
    total = None
    for c in range(0, a.shape[1], 1024):
        part = torch.matmul(a[:, c:c + 1024].float(), b[:, c:c + 1024].float().t())
        total = part.double() if total is None else total.add_(part)
    return total


def _scaled(a, sa, b, sb, dtype):
    return _product(a, b).mul_(sa.double().unsqueeze(1)).mul_(sb.double()).to(dtype)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "product":
        return _scaled(s["a"], s["sa"], s["b"], s["sb"], _dtype(case["out"]))
    if op == "experts":
        N, at = case["N"], s["host"]
        C = torch.zeros(s["a"].shape[0], N, dtype=_dtype(case["out"]), device=DEV)
        for e in range(case["E"]):
            rows, cols = slice(at[e], at[e + 1]), slice(e * N, e * N + N)
            if at[e] < at[e + 1]:
                C[rows] = _scaled(s["a"][rows], s["sa"][rows], s["b"][cols], s["sb"][cols], C.dtype)
        return C
    if op == "quantise":
        codes, scales = _quantise(s["x"])
        values = (codes * scales.double().unsqueeze(1)).to(torch.bfloat16)
        if not case["sort"]:
            return {"values": values, "scales": scales}
        return {"values": _sorted(s, values), "scales": _sorted(s, scales.unsqueeze(1)).squeeze(1), "pos": _positions(s)}
    if op == "dispatch":
        return {"y": _sorted(s, s["x"]), "pos": _positions(s)}
    T, k, w = case["T"], case["k"], s["weights"]
    rows = lambda j: torch.where((s["pos"][j] >= 0).unsqueeze(1), s["y"][s["pos"][j].clamp(min=0)].float(), 0.0)  # noqa: E731
    if op == "combine":
        out = torch.zeros(T, case["cols"], device=DEV)
        for j in range(k):
            out += rows(j) if w is None else w[:, j:j + 1] * rows(j)
        return out.to(s["y"].dtype)
    dout, order = s["dout"].float(), s["order"].long()
    dy = _sorted(s, dout) * w[order % T, order // T].unsqueeze(1)
    dw = torch.stack([(dout * rows(j)).sum(1) for j in range(k)], 1)
    return {"dy": dy.to(s["y"].dtype), "dweights": dw}


# ---- the framework's operators ------------------------------------------------------------------

_lib = None


def _framework():
    global _lib
    if _lib is None:
        from concurrent_gemm_dma_amd import _c3

        _c3.c3_init(0)
        _lib = _c3
    return _lib


def _calls(s):
    c3, case = _framework(), s["case"]
    op = case["op"]
    kind = lambda name: c3.C3_BF16 if name == "bf16" else c3.C3_F32  # noqa: E731
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        c3.c3_i8_gemm(s["a"], s["sa"], s["b"], s["sb"], s["C"], kind(case["out"]), M, N, K, N)
        return s["C"]
    if op == "experts":
        E, N, K, rows = case["E"], case["N"], case["K"], case["T"] * case["k"]
        c3.c3_i8_gemm_experts(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["C"], kind(case["out"]), rows, E,
                              N, K, N)
        return s["C"]
    T, k, E, cols, dtype = case["T"], case["k"], case["E"], case["cols"], kind(case["dtype"])
    if op == "quantise":
        out = {"values": s["values"], "scales": s["scales"]}
        if case["sort"]:
            c3.c3_i8_dispatch(s["x"], dtype, T, cols, cols, s["order"], s["offsets"], k, E, s["codes"], s["scales"],
                              s["pos"])
            out["pos"] = s["pos"]
        else:
            c3.c3_i8_quantize(s["x"], dtype, T, cols, cols, s["codes"], s["scales"])
        c3.c3_i8_dequantize(s["codes"], s["scales"], T * k, cols, s["values"], c3.C3_BF16, cols)
        return out
    if op == "dispatch":
        c3.c3_dispatch(s["x"], dtype, T, cols, cols, s["order"], s["offsets"], k, E, s["y"], cols, s["pos"])
        return {"y": s["y"], "pos": s["pos"]}
    if op == "combine":
        c3.c3_combine(s["y"], dtype, T, k, cols, cols, s["pos"], s["weights"], s["out"], cols)
        return s["out"]
    c3.c3_combine_backward(s["dout"], dtype, T, k, cols, cols, s["y"], cols, s["pos"], s["weights"], s["dy"], cols,
                           s["dweights"])
    return {"dy": s["dy"], "dweights": s["dweights"]}


def run(state):
    return _calls(state) if own else _plain(state)


# ---- definitions in 64 bits ---------------------------------------------------------------------


def _exact_quantise(s):
    case = s["case"]
    T, x = case["T"], s["x"].double()
    a = torch.maximum(x.max(1).values, -x.min(1).values).clamp(min=SMALLEST)
    r = (127.0 / a).float().double()  # the definition rounds it to fp32
    values, scales = (x * r[:, None]).round_() * (a / 127.0)[:, None], a / 127.0
    if not case["sort"]:
        return {"values": values, "scales": scales}
    n = int(s["offsets"][-1])
    t = s["order"][:n].long() % T
    out = {"values": torch.zeros(T * case["k"], case["cols"], dtype=torch.float64, device=DEV),
           "scales": torch.zeros(T * case["k"], dtype=torch.float64, device=DEV), "pos": None}
    out["values"][:n], out["scales"][:n] = values[t], scales[t]
    return out


def _exact_experts(s):
    N = s["case"]["N"]
    C = torch.zeros(s["a"].shape[0], N, dtype=torch.float64, device=DEV)
    for e, (lo, hi) in enumerate(zip(s["host"], s["host"][1:])):
        A = s["a"][lo:hi].double() * s["sa"][lo:hi, None].double()
        B = s["b"][e * N:e * N + N].double() * s["sb"][e * N:e * N + N, None].double()
        C[lo:hi] = A @ B.t()
    return C


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "product":
        return (s["a"].double() * s["sa"][:, None].double()) @ (s["b"].double() * s["sb"][:, None].double()).t()
    if op == "experts":
        return _exact_experts(s)
    if op == "quantise":
        return _exact_quantise(s)
    # what follows goes by the rows of the present slots: token and choice of each
    T, k, cols = case["T"], case["k"], case["cols"]
    n = int(s["offsets"][-1])
    slot = s["order"][:n].long()
    t, j = slot % T, slot // T
    if op == "dispatch":
        y = torch.zeros(T * k, cols, dtype=torch.float64, device=DEV)
        y[:n] = s["x"][t].double()
        return {"y": y, "pos": None}
    if op == "combine":
        out = torch.zeros(T, cols, dtype=torch.float64, device=DEV)
        for c in range(k):
            r = (j == c).nonzero().squeeze(1)  # at most one row a token
            y = s["y"][r].double()
            out[t[r]] += y if s["weights"] is None else s["weights"][t[r], c, None].double() * y
        return out
    dy = torch.zeros(T * k, cols, dtype=torch.float64, device=DEV)
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for r in torch.arange(n, device=DEV).split(16384):
        g = s["dout"][t[r]].double()
        dy[r] = g * s["weights"][t[r], j[r], None].double()
        dw[t[r], j[r]] = (g * s["y"][r].double()).sum(1)
    return {"dy": dy, "dweights": dw}
