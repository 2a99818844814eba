"""Host-only checks of the expert-layer entry points: refusals that need no device, operand sizes,
struct layout, and the tests' own 64-bit definitions against differences and closed cases."""
import ctypes

import numpy as np
import pytest

import layer_ref as ref
from concurrent_gemm_dma_amd import _c3 as c3

P = 1 << 20  # an aligned address; nothing here reads it


def refused(status, word, name, *args):
    got = c3.call(name, *args)
    assert got == status, (name, got, c3.c3_last_error())
    assert word in c3.c3_last_error(), c3.c3_last_error()


def opts(**kw):
    return ctypes.byref(c3.route_opts(**{"top_k": 2, **kw}))


def test_mx4_bytes():
    assert c3.c3_mx4_bytes(3, 1) == (3 * 128, 3 * 8)
    assert c3.c3_mx4_bytes(5, 256) == (5 * 128, 5 * 8)
    assert c3.c3_mx4_bytes(5, 257) == (5 * 256, 5 * 16)
    assert c3.c3_mx4_bytes(0, 32) == (0, 0)
    for rows, cols in ((-1, 32), (1, 0), (1, -5), (1, 1 << 31), (1 << 31, 1)):
        with pytest.raises(c3.C3Error):
            c3.c3_mx4_bytes(rows, cols)


def test_route_opts_layout():
    assert ctypes.sizeof(c3.c3_route_opts) == 32


@pytest.mark.parametrize("word,E,ld,kw", [
    ("n_experts", 0, 8, {}), ("n_experts", 1025, 2000, {}), ("ld", 8, 7, {}),
    ("top_k", 8, 8, {"top_k": 0}), ("top_k", 8, 8, {"top_k": 9}), ("top_k", 256, 256, {"top_k": 65}),
    ("n_groups", 8, 8, {"n_groups": 3}), ("n_groups", 8, 8, {"n_groups": 0}),
    ("n_groups", 130, 130, {"n_groups": 65}), ("top_groups", 8, 8, {"n_groups": 4, "top_groups": 5}),
    ("top_groups", 8, 8, {"top_groups": 0}), ("group_top", 8, 8, {"group_top": 3}),
    ("score", 8, 8, {"score": 2}), ("scale", 8, 8, {"scale": float("nan")}),
])
def test_route_refusals(word, E, ld, kw):
    refused(c3.C3_E_INVALID, word, "c3_route", P, c3.C3_F32, 4, E, ld, opts(**kw), None, 2 * P, 3 * P, None)
    refused(c3.C3_E_INVALID, word, "c3_route_backward", P, c3.C3_F32, 4, E, ld, opts(**kw), 2 * P, 3 * P,
            4 * P, ld, None)


def test_route_refuses_pointers_and_types():
    r = lambda *a: refused(c3.C3_E_INVALID, a[0], "c3_route", *a[1:])  # noqa: E731
    r("opts", P, c3.C3_F32, 4, 8, 8, None, None, 2 * P, 3 * P, None)
    r("dtype", P, 7, 4, 8, 8, opts(), None, 2 * P, 3 * P, None)
    r("n_tokens", P, c3.C3_F32, -1, 8, 8, opts(), None, 2 * P, 3 * P, None)
    r("logits is NULL", None, c3.C3_F32, 4, 8, 8, opts(), None, 2 * P, 3 * P, None)
    r("idx is NULL", P, c3.C3_F32, 4, 8, 8, opts(), None, None, 3 * P, None)
    r("aligned", P + 2, c3.C3_F32, 4, 8, 8, opts(), None, 2 * P, 3 * P, None)
    r("aligned", P, c3.C3_F32, 4, 8, 8, opts(), None, 2 * P + 1, 3 * P, None)
    refused(c3.C3_E_OVERLAP, "overlaps", "c3_route", P, c3.C3_F32, 4, 8, 8, opts(), None, P + 64, 3 * P, None)
    refused(c3.C3_E_OVERLAP, "overlaps", "c3_route", P, c3.C3_F32, 4, 8, 8, opts(), None, 2 * P, 2 * P, None)
    refused(c3.C3_E_OVERLAP, "overlaps", "c3_route_backward", P, c3.C3_F32, 4, 8, 8, opts(), 2 * P, 3 * P, P, 8, None)
    refused(c3.C3_E_INVALID, "ld_d", "c3_route_backward", P, c3.C3_F32, 4, 8, 8, opts(), 2 * P, 3 * P, 4 * P, 7, None)


def test_plan_refusals():
    r = lambda word, *a: refused(c3.C3_E_INVALID, word, "c3_route_plan", *a)  # noqa: E731
    r("n_experts", P, 4, 2, 0, 2 * P, 3 * P, None)
    r("n_experts", P, 4, 2, 1025, 2 * P, 3 * P, None)
    r("top_k", P, 4, 0, 8, 2 * P, 3 * P, None)
    r("top_k", P, 4, 65, 8, 2 * P, 3 * P, None)
    r("n_tokens", P, -1, 2, 8, 2 * P, 3 * P, None)
    r("n_tokens", P, 1 << 30, 2, 8, 2 * P, 3 * P, None)
    r("offsets is NULL", P, 4, 2, 8, 2 * P, None, None)
    refused(c3.C3_E_OVERLAP, "overlaps", "c3_route_plan", P, 4, 2, 8, P, 3 * P, None)


def test_quantise_refusals():
    q = lambda word, *a: refused(c3.C3_E_INVALID, word, "c3_mx4_quantize", *a)  # noqa: E731
    q("dtype", P, 2, 4, 64, 64, 0, 0, 2 * P, 3 * P, None)
    q("rows", P, 0, -1, 64, 64, 0, 0, 2 * P, 3 * P, None)
    q("ld", P, 0, 4, 64, 63, 0, 0, 2 * P, 3 * P, None)
    q("ld", P, 0, 4, 64, 1 << 31, 0, 0, 2 * P, 3 * P, None)
    q("transpose", P, 0, 4, 64, 64, 2, 0, 2 * P, 3 * P, None)
    q("rule", P, 0, 4, 64, 64, 0, 2, 2 * P, 3 * P, None)
    q("codes", P, 0, 4, 64, 64, 0, 0, 2 * P + 8, 3 * P, None)
    q("scales", P, 0, 4, 64, 64, 0, 0, 2 * P, 3 * P + 8, None)
    q("x must be", P + 1, 0, 4, 64, 64, 0, 0, 2 * P, 3 * P, None)
    refused(c3.C3_E_OVERLAP, "overlaps", "c3_mx4_quantize", P, 0, 4, 64, 64, 0, 0, P + 256, 3 * P, None)
    d = lambda word, *a: refused(c3.C3_E_INVALID, word, "c3_mx4_dequantize", *a)  # noqa: E731
    d("dtype", P, 2 * P, 4, 64, 3 * P, 5, 64, None)
    d("ld", P, 2 * P, 4, 64, 3 * P, 0, 10, None)
    d("y is NULL", P, 2 * P, 4, 64, None, 0, 64, None)


def test_product_refusals():
    g = lambda word, *a: refused(c3.C3_E_INVALID, word, "c3_mx4_gemm", *a)  # noqa: E731
    g("dtype", P, 2 * P, 3 * P, 4 * P, 5 * P, 9, 8, 8, 64, 8, None)
    g("K in", P, 2 * P, 3 * P, 4 * P, 5 * P, 0, 8, 8, 0, 8, None)
    g("M, N", P, 2 * P, 3 * P, 4 * P, 5 * P, 0, -1, 8, 64, 8, None)
    g("M, N", P, 2 * P, 3 * P, 4 * P, 5 * P, 0, (1 << 21) + 1, 8, 64, 8, None)
    g("ldc", P, 2 * P, 3 * P, 4 * P, 5 * P, 0, 8, 8, 64, 7, None)
    g("A must be", P + 4, 2 * P, 3 * P, 4 * P, 5 * P, 0, 8, 8, 64, 8, None)
    g("sB is NULL", P, 2 * P, 3 * P, None, 5 * P, 0, 8, 8, 64, 8, None)
    refused(c3.C3_E_OVERLAP, "overlaps", "c3_mx4_gemm", P, 2 * P, 3 * P, 4 * P, P, 0, 8, 8, 64, 8, None)


def test_experts_refusals():
    def x(word, status=c3.C3_E_INVALID, a_rows=8, dtype=0, T=8, k=2, E=4, N=16, K=64, ldc=16, C=9 * P):
        refused(status, word, "c3_mx4_gemm_experts", P, 2 * P, a_rows, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, C,
                dtype, T, k, E, N, K, ldc, None)

    x("dtype", dtype=2)
    x("n_experts", E=0)
    x("n_experts", E=1025)
    x("top_k", k=0)
    x("n_tokens", T=-1)
    x("n_tokens", T=1 << 24)
    x("a_rows", a_rows=9)
    x("K in", K=0)
    x("ldc", ldc=15)
    x("C is NULL", C=None)
    x("overlaps", status=c3.C3_E_OVERLAP, C=7 * P)
    x("4 GiB", status=c3.C3_E_UNSUPPORTED, T=1 << 20, a_rows=1 << 20, K=1 << 20)


def test_valid_calls_need_init():
    assert c3.call("c3_mx4_gemm", P, 2 * P, 3 * P, 4 * P, 5 * P, 0, 8, 8, 64, 8, None) == c3.C3_E_NOT_INIT
    assert c3.call("c3_mx4_gemm", P, 2 * P, 3 * P, 4 * P, 5 * P, 0, 0, 8, 64, 8, None) == c3.C3_E_NOT_INIT
    assert c3.call("c3_route", P, 1, 4, 8, 8, opts(), None, 2 * P, 3 * P, None) == c3.C3_E_NOT_INIT


def test_definition_codes_closed_cases():
    x = np.zeros((1, 32), np.float32)
    x[0, :9] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -7.9]
    codes, scales = ref.quantize(x)
    n = np.stack((codes & 15, codes >> 4), -1).reshape(-1)[:9]
    # unit 1; ties go to the even code, 5 to 4, 7.9 saturates
    assert scales[0, 0] == 127 and list(n) == [6, 0, 2, 2, 4, 4, 6, 6, 15]
    assert ref.quantize(x, up=True)[1][0, 0] == 128
    x[0, 3] = np.inf
    codes, scales = ref.quantize(x)
    assert scales[0, 0] == 255 and not codes.any()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_definition_gradient_against_differences(kind, renorm):
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1.5, (6, 10))
    x[0, 3] = -np.inf
    idx, _ = ref.route(x, 3, kind, renorm=renorm)
    idx[1, 2] = -1
    dw = rng.normal(0, 1, idx.shape)
    d, _ = ref.route_gradient(x, idx, dw, kind, renorm, scale=1.5)
    h = 1e-5
    for t in range(6):
        at = idx[t][idx[t] >= 0]
        for e in range(10):
            if np.isneginf(x[t, e]):
                continue
            lo, hi = x[t].copy(), x[t].copy()
            lo[e] -= h
            hi[e] += h
            f = [(dw[t, :len(at)] * ref.weights_of(ref.clean(y), at, kind, renorm, 1.5)).sum() for y in (lo, hi)]
            # central difference: truncation below h^2 * 10, rounding below 1e-15 / h
            assert abs((f[1] - f[0]) / (2 * h) - d[t, e]) < 1e-9 + 1e-15 / h


@pytest.mark.parametrize("top_k", [1, 2, 3, 5, 7, 64])
def test_plan_takes_every_number_of_slots_below_its_limit(top_k):
    """n_tokens * top_k < 2^31, whether top_k divides 2^31 or not."""
    at = [n << 40 for n in (1, 2, 3)]
    most = ((1 << 31) - 1) // top_k
    assert c3.call("c3_route_plan", at[0], most, top_k, 8, at[1], at[2], None) == c3.C3_E_NOT_INIT
    refused(c3.C3_E_INVALID, "n_tokens", "c3_route_plan", at[0], most + 1, top_k, 8, at[1], at[2], None)
