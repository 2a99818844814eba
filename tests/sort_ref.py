"""Plain 64-bit definitions of sorting rows by expert, of the way back and of int8 operands, in
numpy, for the tests. Nothing here is shared with the library."""
import numpy as np

from layer_ref import bf16_round, plan  # noqa: F401

HALF = {0: 2.0 ** -8, 1: 2.0 ** -24}  # half a step of bf16 and fp32, relative
TINY = 2.0 ** -133  # above half the distance of bf16's and fp32's smallest values


def padded(cols):
    return -(-cols // 128) * 128


def positions(order, n, S):
    """pos of every slot named by order, -1 without a row; -2 where order names it not."""
    pos = np.full(S, -2, np.int32)
    for p, s in enumerate(order):
        if 0 <= s < S:
            pos[s] = p if p < n else -1
    return pos


def sort_rows(x, order, n):
    """Rows [n][cols] of x [T][cols]."""
    return x[order[:n] % x.shape[0]]


def combine(y, pos, w):
    """(out, bound on fp32's error) of y [S][cols], pos [k][T], w [T][k] or None: one rounding of a
    fused multiply and add for each choice, of a sum no larger than the terms' magnitudes."""
    k, T = pos.shape
    out = np.zeros((T, y.shape[1]))
    size = np.zeros_like(out)
    for j in range(k):
        here = (pos[j] >= 0) & (pos[j] < len(y))
        term = y[pos[j][here]].astype(np.float64)
        if w is not None:
            term = term * w[here, j][:, None].astype(np.float64)
        out[here] += term
        size[here] += np.abs(term)
    return out, 1.01 * k * 2.0 ** -24 * size + TINY


def combine_gradient(dout, y, pos, w):
    """(dy [S][cols], rows it writes, dw [T][k], bound of dw: a sum in fp32 in any order)."""
    k, T = pos.shape
    S, cols = y.shape
    d = dout.astype(np.float64)
    dy, written = np.zeros((S, cols)), np.zeros(S, bool)
    dw, bound = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        here = (pos[j] >= 0) & (pos[j] < S)
        p = pos[j][here]
        written[p] = True
        dy[p] = d[here] * (1.0 if w is None else w[here, j][:, None].astype(np.float64))
        terms = d[here] * y[p].astype(np.float64)
        dw[here, j] = terms.sum(1)
        bound[here, j] = 1.01 * (cols + 16) * 2.0 ** -24 * np.abs(terms).sum(1)
    return dy, written, dw, bound + cols * 2.0 ** -149


def quantize(x):
    """(codes [rows][P] int8, scales float32) of float32 x [rows][cols]."""
    rows, cols = x.shape
    a = np.abs(x).max(1) if cols else np.zeros(rows, np.float32)
    bad = ~np.isfinite(a)
    a = np.maximum(np.where(bad, np.float32(1), a), np.float32(2.0 ** -119)).astype(np.float32)
    r = (np.float32(127) / a).astype(np.float64)
    n = np.rint(np.where(bad[:, None], 0.0, x).astype(np.float64) * r[:, None])  # 48 bits: exact
    codes = np.zeros((rows, padded(cols)), np.int8)
    codes[:, :cols] = n
    return codes, np.where(bad, np.float32(np.nan), (a / np.float32(127)).astype(np.float32))


def rounded(x, dtype):
    return bf16_round(x) if dtype == 0 else np.asarray(x, np.float32)


def product(A, sA, B, sB):
    """float32 sA[m] * sB[n] * sums of codes: exact sums, then three roundings, as defined."""
    total = A.astype(np.float64) @ B.astype(np.float64).T  # below 2^31: exact in any order
    with np.errstate(all="ignore"):
        return (total.astype(np.float32) * sA[:, None].astype(np.float32)) * sB.astype(np.float32)
