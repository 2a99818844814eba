"""Plain 64-bit definitions of what the expert-layer entry points compute, in numpy, for the tests.

Nothing here is shared with the library. Operands are (codes, scales) uint8 arrays in the layout
include/c3.h states; values are float64.
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
LARGEST = float(np.finfo(np.float32).max)


def padded(cols):
    return -(-cols // 256) * 256


def bf16_round(x):
    """float32 nearest-even bf16 values of an array (finite)."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)).view(np.float32)


def quantize(x, up=False):
    """(codes, scales) of float32 x [rows][cols]."""
    rows, cols = x.shape
    P = padded(cols)
    b = np.zeros((rows, P))
    b[:, :cols] = x
    b = b.reshape(rows, P // 32, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    amax = np.where(bad, 1.0, amax)
    e = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1.0))[1] - 3, -127)
    if up:
        e = e + (amax > 6.0 * np.exp2(e.astype(float)))
    e = np.maximum(e, -127)
    y = np.where(bad[..., None], 0.0, b) / np.exp2(e.astype(float))[..., None]
    d = np.abs(np.minimum(np.abs(y), 6.0)[..., None] - GRID)
    least = d.min(-1, keepdims=True)
    near = d == least  # one, or two at a tie: then the even code
    first = near.argmax(-1)
    last = 7 - near[..., ::-1].argmax(-1)
    code = np.where((first != last) & (first % 2 == 1), last, first) + 8 * np.signbit(y)
    code = np.where(bad[..., None], 0, code).reshape(rows, P).astype(np.uint8)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def values(codes, scales, cols):
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127))
    v = GRID[n & 7] * np.where(n & 8, -1.0, 1.0)
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(v.shape)[..., :cols]


def product(A, B):
    """(A . B^T, bound on the error of adding its terms up in fp32 in any order)."""
    K = A.shape[-1]
    return A @ B.T, (K + 16) * 2.0 ** -24 * (np.abs(A) @ np.abs(B).T)


def scores(l, kind):
    """Scores of one token's logits (float64, -inf where out of reach)."""
    reach = l > -np.inf
    s = np.zeros_like(l)
    if kind == "sigmoid":
        x = l[reach]
        t = np.exp(-np.abs(x))
        s[reach] = np.where(x >= 0, 1 / (1 + t), t / (1 + t))
    elif reach.any():
        p = np.exp(l[reach] - l[reach].max())
        s[reach] = p / p.sum()
    return s


def clean(x):
    l = np.minimum(x.astype(np.float64), LARGEST)
    return np.where(np.isnan(l), -np.inf, l)


def weights_of(l, chosen, kind, renorm, scale=1.0):
    """Weights of the chosen experts of one token, from logarithms where a sum divides."""
    if not len(chosen):
        return np.zeros(0)
    if not renorm:
        return scores(l, kind)[chosen] * scale
    log = -np.logaddexp(0, -l[chosen]) if kind == "sigmoid" else l[chosen]
    log = log - log.max()  # before the sum: logits of 1e38 swallow a log of 2
    return np.exp(log - np.logaddexp.reduce(log)) * scale


def route(x, k, kind="softmax", groups=1, top_groups=1, group_top=1, bias=None, renorm=True,
          scale=1.0):
    """(idx, weights) of logits x [T][E]."""
    T, E = x.shape
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        l = clean(x[t])
        s = scores(l, kind)
        v = l.copy() if bias is None else np.where(l > -np.inf, s + bias.astype(np.float64), -np.inf)
        v[np.isnan(v)] = -np.inf
        if groups > 1:
            size = E // groups
            worth = []
            for g in range(groups):
                mine = sorted((e for e in range(g * size, (g + 1) * size) if v[e] > -np.inf),
                              key=lambda e: (-v[e], e))[:group_top]
                if group_top == 1:
                    worth.append(v[mine[0]] if mine else -np.inf)
                else:
                    b = 0.0 if bias is None else bias[mine].astype(np.float64)
                    worth.append((s[mine] + b).sum() if mine else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            v = np.where(np.isin(np.arange(E) // size, kept), v, -np.inf)
        chosen = [e for e in sorted(range(E), key=lambda e: (-v[e], e))[:k] if v[e] > -np.inf]
        idx[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = weights_of(l, np.array(chosen, int), kind, renorm, scale)
    return idx, w


def route_gradient(x, idx, dw, kind="softmax", renorm=True, scale=1.0):
    """d/dlogits of sum(dw * weights), the choice held fixed; and the size of its terms."""
    T, E = x.shape
    d = np.zeros((T, E))
    size = np.zeros((T, E))
    for t in range(T):
        l = clean(x[t])
        use = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E and l[idx[t, j]] > -np.inf]
        at = idx[t, use]
        g = dw[t, use].astype(np.float64) * scale
        if not len(at):
            continue
        if renorm:
            w = weights_of(l, at, kind, True)
            inner, most = (g * w).sum(), (np.abs(g) * w).sum()
            f = 1 / (1 + np.exp(np.minimum(l[at], 700))) if kind == "sigmoid" else 1.0
            np.add.at(d[t], at, w * (g - inner) * f)
            np.add.at(size[t], at, w * (np.abs(g) + most) * f)
        elif kind == "sigmoid":
            s = scores(l, kind)[at]
            f = g * s * (1 / (1 + np.exp(np.minimum(l[at], 700))))
            np.add.at(d[t], at, f)
            np.add.at(size[t], at, np.abs(f))
        else:
            p = scores(l, kind)
            inner, most = (g * p[at]).sum(), (np.abs(g) * p[at]).sum()
            d[t] -= p * inner
            size[t] += p * most
            np.add.at(d[t], at, p[at] * g)
            np.add.at(size[t], at, p[at] * np.abs(g))
    return d, size


def plan(idx, E):
    T, k = idx.shape
    e = np.where((idx >= 0) & (idx < E), idx, E).reshape(-1)
    at = np.argsort(e, kind="stable")
    order = (at % k * T + at // k).astype(np.int32)
    return order, np.searchsorted(e[at], np.arange(E + 1)).astype(np.int32)
