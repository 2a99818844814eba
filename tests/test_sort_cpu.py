"""Host-only checks of the entry points for sorted rows and int8 operands: refusals that need no
device, sizes, and the tests' own definitions against closed cases and differences."""
import numpy as np
import pytest

import sort_ref as ref
from concurrent_gemm_dma_amd import _c3 as c3

P = 1 << 20  # an aligned address; nothing here reads it


def refused(status, word, name, *args):
    got = c3.call(name, *args)
    assert got == status, (name, got, c3.c3_last_error())
    assert word in c3.c3_last_error(), c3.c3_last_error()


BAD = {c3.C3_E_OVERLAP: "overlaps", c3.C3_E_NOT_INIT: "c3_init"}


def dispatch(word, status=c3.C3_E_INVALID, name="c3_dispatch", x=P, dtype=0, T=4, cols=64, ld=64, order=2 * P,
             offsets=3 * P, k=2, E=8, y=4 * P, ld_y=64, pos=5 * P, scales=6 * P):
    if name == "c3_dispatch":
        refused(status, word, name, x, dtype, T, cols, ld, order, offsets, k, E, y, ld_y, pos, None)
    else:
        refused(status, word, name, x, dtype, T, cols, ld, order, offsets, k, E, y, scales, pos, None)


@pytest.mark.parametrize("name", ["c3_dispatch", "c3_i8_dispatch"])
def test_dispatch_refusals(name):
    d = lambda word, status=c3.C3_E_INVALID, **kw: dispatch(word, status, name, **kw)  # noqa: E731
    d("dtype", dtype=2)
    d("top_k", k=0)
    d("top_k", k=65)
    d("n_tokens", T=-1)
    d("n_tokens", T=1 << 30)
    d("n_experts", E=0)
    d("n_experts", E=1025)
    d("cols", cols=0)
    d("cols", cols=1 << 31, ld=1 << 31)
    d("ld", ld=63)
    d("ld", ld=1 << 31)
    d("x is NULL", x=None)
    d("order is NULL", order=None)
    d("offsets is NULL", offsets=None)
    d("pos is NULL", pos=None)
    d("x must be", x=P + 1)
    d("x must be", x=P + 2, dtype=1)
    d("order must be", order=2 * P + 2)
    d("overlaps", c3.C3_E_OVERLAP, y=P)
    d("overlaps", c3.C3_E_OVERLAP, pos=2 * P)
    d("overlaps", c3.C3_E_OVERLAP, pos=4 * P)
    d("c3_init", c3.C3_E_NOT_INIT)
    d("c3_init", c3.C3_E_NOT_INIT, T=0)
    if name == "c3_dispatch":
        d("ld_y", ld_y=63)
        d("y is NULL", y=None)
        d("y must be", y=4 * P + 1)
    else:
        d("codes is NULL", y=None)
        d("codes must be", y=4 * P + 8)
        d("scales must be", scales=6 * P + 2)
        d("overlaps", c3.C3_E_OVERLAP, scales=4 * P)


def test_combine_refusals():
    def c(word, status=c3.C3_E_INVALID, y=P, dtype=0, T=4, k=2, cols=64, ld_y=64, pos=2 * P, w=3 * P, out=4 * P, ld=64):
        refused(status, word, "c3_combine", y, dtype, T, k, cols, ld_y, pos, w, out, ld, None)

    c("dtype", dtype=-1)
    c("n_tokens", T=1 << 30)
    c("top_k", k=0)
    c("cols", cols=0)
    c("ld_y", ld_y=63)
    c("ld_out", ld=63)
    c("y is NULL", y=None)
    c("pos is NULL", pos=None)
    c("out is NULL", out=None)
    c("weights must be", w=3 * P + 2)
    c("overlaps", c3.C3_E_OVERLAP, out=P)
    c("overlaps", c3.C3_E_OVERLAP, out=3 * P)
    c("c3_init", c3.C3_E_NOT_INIT, w=None)


def test_combine_backward_refusals():
    def c(word, status=c3.C3_E_INVALID, dout=P, dtype=0, T=4, k=2, cols=64, ld=64, y=2 * P, ld_y=64, pos=3 * P,
          w=4 * P, dy=5 * P, ld_dy=64, dw=6 * P):
        refused(status, word, "c3_combine_backward", dout, dtype, T, k, cols, ld, y, ld_y, pos, w, dy, ld_dy, dw, None)

    c("dtype", dtype=2)
    c("n_tokens", T=-1)
    c("top_k", k=65)
    c("cols", cols=0)
    c("ld_d", ld=63)
    c("ld_y", ld_y=63)
    c("ld_dy", ld_dy=63)
    c("dout is NULL", dout=None)
    c("y is NULL", y=None)
    c("pos is NULL", pos=None)
    c("dy is NULL", dy=None)
    c("overlaps", c3.C3_E_OVERLAP, dy=P)
    c("overlaps", c3.C3_E_OVERLAP, dy=2 * P)
    c("overlaps", c3.C3_E_OVERLAP, dw=4 * P)
    c("c3_init", c3.C3_E_NOT_INIT, y=None, dw=None, ld_y=0)


def test_i8_bytes():
    assert c3.c3_i8_bytes(3, 1) == (3 * 128, 12)
    assert c3.c3_i8_bytes(5, 128) == (5 * 128, 20)
    assert c3.c3_i8_bytes(5, 129) == (5 * 256, 20)
    assert c3.c3_i8_bytes(0, 32) == (0, 0)
    for rows, cols in ((-1, 32), (1, 0), (1, -5), (1, 1 << 31), (1 << 31, 1)):
        with pytest.raises(c3.C3Error):
            c3.c3_i8_bytes(rows, cols)


def test_quantise_refusals():
    q = lambda word, *a: refused(c3.C3_E_INVALID, word, "c3_i8_quantize", *a)  # noqa: E731
    q("dtype", P, 2, 4, 64, 64, 2 * P, 3 * P, None)
    q("rows", P, 0, -1, 64, 64, 2 * P, 3 * P, None)
    q("rows", P, 0, 1 << 31, 64, 64, 2 * P, 3 * P, None)
    q("cols", P, 0, 4, 0, 64, 2 * P, 3 * P, None)
    q("ld", P, 0, 4, 64, 63, 2 * P, 3 * P, None)
    q("x is NULL", None, 0, 4, 64, 64, 2 * P, 3 * P, None)
    q("x must be", P + 1, 0, 4, 64, 64, 2 * P, 3 * P, None)
    q("codes must be", P, 0, 4, 64, 64, 2 * P + 8, 3 * P, None)
    q("scales is NULL", P, 0, 4, 64, 64, 2 * P, None, None)
    refused(c3.C3_E_OVERLAP, "overlaps", "c3_i8_quantize", P, 0, 4, 64, 64, P + 256, 3 * P, None)
    refused(c3.C3_E_NOT_INIT, "c3_init", "c3_i8_quantize", P, 0, 0, 64, 64, 2 * P, 3 * P, None)
    d = lambda word, *a: refused(c3.C3_E_INVALID, word, "c3_i8_dequantize", *a)  # noqa: E731
    d("dtype", P, 2 * P, 4, 64, 3 * P, 5, 64, None)
    d("cols", P, 2 * P, 4, 0, 3 * P, 0, 64, None)
    d("ld", P, 2 * P, 4, 64, 3 * P, 0, 10, None)
    d("y is NULL", P, 2 * P, 4, 64, None, 0, 64, None)
    d("codes must be", P + 4, 2 * P, 4, 64, 3 * P, 0, 64, None)
    refused(c3.C3_E_OVERLAP, "overlaps", "c3_i8_dequantize", P, 2 * P, 4, 64, P, 0, 64, None)


def test_product_refusals():
    def g(word, status=c3.C3_E_INVALID, A=P, sA=2 * P, B=3 * P, sB=4 * P, C=5 * P, dtype=0, M=8, N=8, K=64, ldc=8):
        refused(status, word, "c3_i8_gemm", A, sA, B, sB, C, dtype, M, N, K, ldc, None)

    g("dtype", dtype=9)
    g("M must", M=-1)
    g("M must", M=(1 << 21) + 1)
    g("N must", N=(1 << 21) + 1, ldc=1 << 22)
    g("K must", K=0)
    g("K must", K=c3.C3_I8_MAX_K + 1)
    g("ldc", ldc=7)
    g("A must be", A=P + 4)
    g("sB is NULL", sB=None)
    g("overlaps", c3.C3_E_OVERLAP, C=P)
    g("c3_init", c3.C3_E_NOT_INIT, K=c3.C3_I8_MAX_K)
    g("c3_init", c3.C3_E_NOT_INIT, M=0)


def test_experts_refusals():
    def x(word, status=c3.C3_E_INVALID, dtype=0, rows=16, E=4, N=16, K=64, ldc=16, offsets=5 * P, C=9 * P):
        refused(status, word, "c3_i8_gemm_experts", P, 2 * P, 3 * P, 4 * P, offsets, C, dtype, rows, E, N, K, ldc, None)

    x("dtype", dtype=2)
    x("n_experts", E=0)
    x("n_experts", E=1025)
    x("n_rows", rows=-1)
    x("n_rows", rows=(1 << 24) + 1)
    x("N must", N=-1)
    x("K must", K=c3.C3_I8_MAX_K + 1)
    x("ldc", ldc=15)
    x("offsets is NULL", offsets=None)
    x("C is NULL", C=None)
    x("overlaps", c3.C3_E_OVERLAP, C=5 * P)
    x("c3_init", c3.C3_E_NOT_INIT)
    x("c3_init", c3.C3_E_NOT_INIT, rows=0)


@pytest.mark.parametrize("top_k", [1, 2, 3, 7, 64])
def test_every_number_of_slots_below_its_limit(top_k):
    at = [n << 44 for n in range(1, 6)]
    most = ((1 << 31) - 1) // top_k
    args = lambda T: (at[0], 0, T, 64, 64, at[1], at[2], top_k, 8, at[3], 64, at[4], None)  # noqa: E731
    assert c3.call("c3_dispatch", *args(most)) == c3.C3_E_NOT_INIT
    refused(c3.C3_E_INVALID, "n_tokens", "c3_dispatch", *args(most + 1))


def test_definition_codes_closed_cases():
    x = np.zeros((5, 6), np.float32)
    x[0] = [127, 0.5, 1.5, -2.5, -0.5, 126.5]  # unit 1: ties go to the even code
    x[1, 2] = np.inf
    x[2, 3] = -1e-45
    codes, scales = ref.quantize(x)
    assert codes.shape == (5, 128) and not codes[:, 6:].any()
    assert list(codes[0, :6]) == [127, 0, 2, -2, 0, 126] and scales[0] == 1.0
    assert np.isnan(scales[1]) and not codes[1].any()
    assert not codes[2:].any() and (scales[2:] == np.float32(2.0 ** -119) / np.float32(127)).all()


def test_definition_gradient_against_differences():
    """d of sum(g * out) over y and the weights, by differences (out is linear in each: exact but
    for rounding)."""
    rng = np.random.default_rng(4)
    T, k, cols, E = 7, 3, 5, 4
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    idx[2] = -1
    order, offsets = ref.plan(idx, E)
    n = offsets[-1]
    pos = ref.positions(order, n, T * k).reshape(k, T)
    assert sorted(pos[pos >= 0]) == list(range(n)) and (pos[:, 2] == -1).all()
    y, w, g = rng.normal(size=(T * k, cols)), rng.normal(size=(T, k)), rng.normal(size=(T, cols))
    f = lambda y, w: (g * ref.combine(y, pos, w)[0]).sum()  # noqa: E731
    dy, written, dw, _ = ref.combine_gradient(g, y, pos, w)
    assert written.sum() == n
    for array, d in ((y, dy), (w, dw)):
        for i in np.ndindex(array.shape):
            was = array[i]
            array[i] = was + 0.5
            hi = f(y, w)
            array[i] = was - 0.5
            lo = f(y, w)
            array[i] = was
            # 105 terms below 40, rounded to 53 bits
            assert abs(hi - lo - d[i]) < 105 * 40 * 2.0 ** -52 * 4
    # the sort's gradient: the combination without weights
    x = rng.normal(size=(T, cols))
    gy = rng.normal(size=(T * k, cols))
    dx = ref.combine(gy, pos, None)[0]
    at = lambda x: (gy[:n] * ref.sort_rows(x, order, n)).sum()  # noqa: E731
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += 0.5
        lo[i] -= 0.5
        assert abs(at(hi) - at(lo) - dx[i]) < 105 * 40 * 2.0 ** -52 * 4
