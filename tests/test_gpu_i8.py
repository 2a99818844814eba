"""int8 operands and their products on the GPU against the definitions of sort_ref, bit for bit:
codes, scales, values and products (exact sums, then the roundings that the header states)."""
import numpy as np
import pytest

import sort_ref as ref
from test_gpu_sort import CANARY, Rows, dev, routing, sync, values

pytestmark = pytest.mark.gpu


def wide(rng, rows, cols, dtype):
    """Rows over the whole exponent range, zeros, subnormals and rows that are all zero among them."""
    x = rng.normal(0, 1, (rows, cols)) * np.exp2(rng.integers(-146, 127, (rows, 1)).astype(float))
    x *= np.exp2(rng.integers(-9, 1, (rows, cols)).astype(float))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    x[rng.random(rows) < 0.1] = 0.0
    x = np.clip(x, -3e38, 3e38).astype(np.float32)
    return ref.bf16_round(x) if dtype == 0 else x


def quantise(c3, x, dtype, ld=None, shift=0, stream=None):
    import torch

    rows, cols = x.shape
    X = Rows(rows, cols, dtype, ld, shift, x)
    X.whole.masked_fill_(X.whole == CANARY, float("nan"))  # what is past cols is not read
    nc, ns = c3.c3_i8_bytes(rows, cols)
    codes = torch.full((nc + 64,), 0x5A, dtype=torch.int8, device="cuda:0")
    scales = torch.full((ns // 4 + 16,), CANARY, device="cuda:0")
    X.view()[:] = dev(x).to(X.whole.dtype)
    c3.c3_i8_quantize(X.ptr(), dtype, rows, cols, X.ld, codes, scales, stream)
    sync()
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    assert (codes[nc:] == 0x5A).all() and (scales[rows:] == CANARY).all()
    return codes[:nc].reshape(rows, -1), scales[:rows]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,cols,more,shift", [
    (1, 1, 0, 0), (1, 128, 0, 0), (3, 127, 0, 1), (2, 129, 3, 0), (5, 1000, 0, 3), (130, 136, 0, 0), (9, 2048, 0, 0),
    (7, 2049, 1, 0), (1, 16384, 0, 0), (40, 16384, 0, 0), (3, 16385, 0, 5), (2, 70001, 0, 0), (1000, 520, 8, 0),
    (5000, 72, 0, 0), (700, 4096, 0, 0), (1, 131072, 0, 0), (50, 400, 0, 0)])
def test_quantise(c3gpu, rows, cols, more, shift, dtype):
    x = wide(np.random.default_rng(rows * 7919 + cols), rows, cols, dtype)
    codes, scales = quantise(c3gpu, x, dtype, cols + more, shift)
    want = ref.quantize(x)
    np.testing.assert_array_equal(scales, want[1])
    np.testing.assert_array_equal(codes, want[0])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("cols", [130, 5000, 20000])
def test_quantise_ties_infinities_and_the_lowest_value(c3gpu, dtype, cols):
    rng = np.random.default_rng(cols)
    x = np.zeros((12, cols), np.float32)
    x[0] = np.arange(cols) % 255 - 127  # whole units
    x[1] = (np.arange(cols) % 253 - 126) + 0.5  # ties, the unit 1 from the row's largest
    x[1, 7] = 127
    x[2] = -x[1] * 2.0 ** -20
    x[3] = np.finfo(np.float32).min if dtype else ref.bf16_round(np.float32(-3.38e38))
    x[4:9] = values(rng, (5, cols), dtype)
    x[4, cols - 1], x[5, 0], x[6, cols // 2] = np.inf, -np.inf, np.nan
    x[7, 3] = np.nan
    x[7, 4] = np.inf
    x[9, 1] = 1e-45 if dtype else 2.0 ** -133
    x[10] = 2.0 ** -119
    x[11, cols - 1] = -5
    if dtype == 0:
        x = np.where(np.isfinite(x), ref.bf16_round(np.where(np.isfinite(x), x, 0)), x)
    codes, scales = quantise(c3gpu, x, dtype)
    want = ref.quantize(x)
    np.testing.assert_array_equal(scales, want[1])
    np.testing.assert_array_equal(codes, want[0])
    assert np.isnan(scales[4:8]).all() and np.isfinite(scales[8:]).all()


def test_quantise_values_next_to_borders(c3gpu):
    """fp32 values at and next to every half unit, for several largest values."""
    rows = []
    for a in (1.0, 127.0, 3.14159, 0.9999999, 2.0 ** -119, 1e38, 97.0):
        a = np.float32(a)
        half = ((np.arange(-126, 127) + 0.5) * (float(a) / 127)).astype(np.float32)
        row = np.concatenate([half, np.nextafter(half, np.float32(np.inf)), np.nextafter(half, np.float32(-np.inf)), [a]])
        rows.append(row[np.abs(row) <= a] if False else np.clip(row, -a, a))
    x = np.stack(rows).astype(np.float32)
    codes, scales = quantise(c3gpu, x, 1)
    want = ref.quantize(x)
    np.testing.assert_array_equal(scales, want[1])
    np.testing.assert_array_equal(codes, want[0])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,E,k,cols,more,shift,masked", [
    (1, 4, 4, 4096, 0, 0, 0.0), (3, 8, 2, 7, 1, 3, 0.0), (8, 32, 4, 16385, 0, 0, 0.0), (17, 5, 3, 129, 0, 1, 0.3),
    (700, 16, 8, 520, 0, 0, 0.1), (6000, 64, 7, 65, 3, 5, 0.05), (1030, 24, 3, 5000, 0, 0, 0.1), (40, 8, 2, 640, 0, 0, 1.0),
    (900, 16, 8, 2048, 0, 0, 0.0), (300, 16, 8, 17000, 0, 0, 0.1), (20, 8, 2, 1500, 0, 0, 0.1), (20, 8, 2, 6000, 0, 0, 0.1),
    (20, 8, 2, 12001, 0, 0, 0.1), (10000, 16, 7, 100, 0, 0, 0.1), (5100, 16, 7, 200, 1, 0, 0.1), (2600, 16, 7, 400, 0, 0, 0.1),
    (600, 16, 3, 4000, 0, 1, 0.1), (150, 16, 3, 16000, 0, 0, 0.1)])
def test_sorted_quantise(c3gpu, T, E, k, cols, more, shift, masked, dtype):
    import torch

    rng = np.random.default_rng(T * 31 + cols)
    order, offsets, n = routing(rng, T, E, k, masked)
    x = wide(rng, T, cols, dtype)
    x[0, cols // 2] = np.nan
    X = Rows(T, cols, dtype, cols + more, shift, x)
    S, P = T * k, ref.padded(cols)
    codes = torch.full((S * P + 64,), 0x5A, dtype=torch.int8, device="cuda:0")
    scales, pos = torch.full((S + 8,), CANARY, device="cuda:0"), torch.full((S + 8,), -9, dtype=torch.int32, device="cuda:0")
    c3gpu.c3_i8_dispatch(X.ptr(), dtype, T, cols, X.ld, dev(order), dev(offsets), k, E, codes, scales, pos)
    sync()
    got = pos.cpu().numpy()
    np.testing.assert_array_equal(got[:S], ref.positions(order, n, S))
    assert (got[S:] == -9).all()
    want = ref.quantize(x)
    t = order[:n] % T
    np.testing.assert_array_equal(scales.cpu().numpy()[:n], want[1][t])
    assert (scales.cpu().numpy()[n:] == CANARY).all()
    got = codes.cpu().numpy()
    np.testing.assert_array_equal(got[:n * P].reshape(n, P), want[0][t])
    assert (got[n * P:] == 0x5A).all()


@pytest.mark.parametrize("T", [9, 3000])
def test_sorted_quantise_skips_what_is_no_slot(c3gpu, T):
    import torch

    rng = np.random.default_rng(2)
    k, E, cols = 3, 8, 300
    order, offsets, n = routing(rng, T, E, k, 0.0)
    S, P = T * k, 384
    bad = rng.random(S) < 0.2
    order = np.where(bad, rng.choice([-1, S, 2 ** 31 - 1, -2 ** 31], S), order).astype(np.int32)
    offsets[-1] = 1 << 30
    x = wide(rng, T, cols, 0)
    X = Rows(T, cols, 0, values=x)
    codes = torch.full((S, P), 0x5A, dtype=torch.int8, device="cuda:0")
    scales, pos = torch.full((S,), CANARY, device="cuda:0"), torch.full((S,), -2, dtype=torch.int32, device="cuda:0")
    c3gpu.c3_i8_dispatch(X.ptr(), 0, T, cols, cols, dev(order), dev(offsets), k, E, codes, scales, pos)
    sync()
    np.testing.assert_array_equal(pos.cpu().numpy(), ref.positions(order, S, S))
    want, got = ref.quantize(x), codes.cpu().numpy()
    np.testing.assert_array_equal(got[~bad], want[0][order[~bad] % T])
    assert (got[bad] == 0x5A).all() and (scales.cpu().numpy()[bad] == CANARY).all()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,cols,more,shift", [(1, 1, 0, 0), (1, 16384, 0, 0), (5, 130, 3, 1), (300, 1001, 0, 0),
                                                  (33, 4096, 8, 0), (4, 9, 0, 7), (2000, 64, 0, 0)])
def test_dequantise(c3gpu, rows, cols, more, shift, dtype):
    rng = np.random.default_rng(rows + cols)
    codes = rng.integers(-128, 128, (rows, ref.padded(cols))).astype(np.int8)  # past cols: not read
    scales = (rng.normal(0, 1, rows) * np.exp2(rng.integers(-120, 120, rows))).astype(np.float32)
    if rows > 4:
        scales[1], scales[2], scales[3] = np.nan, 0.0, np.inf
    y = Rows(rows, cols, dtype, cols + more, shift)
    c3gpu.c3_i8_dequantize(dev(codes), dev(scales), rows, cols, y.ptr(), dtype, y.ld)
    sync()
    y.intact()
    with np.errstate(all="ignore"):
        want = codes[:, :cols].astype(np.float32) * scales[:, None]
        odd = ~np.isfinite(want)
        want = np.where(odd, want, ref.rounded(np.where(odd, 0, want).astype(np.float32), dtype))
    np.testing.assert_array_equal(y.numpy(), want)


def operand(rng, rows, K):
    """Codes over all 256 values with zeros past K, scales of uneven size."""
    codes = np.zeros((rows, ref.padded(K)), np.int8)
    codes[:, :K] = rng.integers(-128, 128, (rows, K))
    return codes, (rng.random(rows) + 0.1).astype(np.float32) * np.exp2(rng.integers(-20, 3, rows)).astype(np.float32)


PRODUCTS = [(1, 1, 1), (1, 28, 64), (1, 4096, 4096), (2, 33, 129), (5, 100, 1000), (16, 64, 128), (16, 512, 8192),
            (17, 31, 257), (33, 130, 384), (64, 2048, 2048), (100, 257, 640), (128, 128, 128), (129, 1000, 300),
            (200, 640, 1024), (256, 256, 256), (257, 255, 512), (300, 5000, 128), (513, 1030, 1152), (777, 4999, 400),
            (1500, 1500, 700), (3000, 64, 2000), (2050, 2300, 900), (1, 20000, 131)]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(c3gpu, M, N, K, dtype):
    rng = np.random.default_rng(M * 101 + N * 7 + K)
    (A, sA), (B, sB) = operand(rng, M, K), operand(rng, N, K)
    more = 3 if N % 2 else 0
    C = Rows(M, N, dtype, N + more, 1 if N % 4 == 1 else 0)
    c3gpu.c3_i8_gemm(dev(A), dev(sA), dev(B), dev(sB), C.ptr(), dtype, M, N, K, C.ld)
    sync()
    C.intact()
    np.testing.assert_array_equal(C.numpy(), ref.rounded(ref.product(A, sA, B, sB), dtype))


def test_product_scales_that_are_no_numbers(c3gpu):
    rng = np.random.default_rng(1)
    M, N, K = 40, 70, 200
    (A, sA), (B, sB) = operand(rng, M, K), operand(rng, N, K)
    A[5] = 0
    sA[3], sA[4], sA[6], sB[9], sB[10] = np.nan, np.inf, 0.0, np.nan, np.float32(3e38)
    C = Rows(M, N, 1)
    c3gpu.c3_i8_gemm(dev(A), dev(sA), dev(B), dev(sB), C.ptr(), 1, M, N, K, N)
    sync()
    np.testing.assert_array_equal(C.numpy(), ref.product(A, sA, B, sB))


@pytest.mark.parametrize("M,N", [(3, 5), (300, 300)])
def test_product_of_the_longest_rows_and_largest_codes(c3gpu, M, N):
    K = c3gpu.C3_I8_MAX_K
    A, B = np.zeros((M, ref.padded(K)), np.int8), np.zeros((N, ref.padded(K)), np.int8)
    A[:, :K], B[:, :K] = -128, -128
    B[1, :K] = 127
    C = Rows(M, N, 1)
    c3gpu.c3_i8_gemm(dev(A), dev(np.ones(M, np.float32)), dev(B), dev(np.ones(N, np.float32)), C.ptr(), 1, M, N, K, N)
    sync()
    want = np.full((M, N), np.float32(K * 16384))
    want[:, 1] = np.float32(-K * 128 * 127)
    np.testing.assert_array_equal(C.numpy(), want)


def test_product_of_operands_past_4_GiB(c3gpu):
    import torch

    rng = np.random.default_rng(5)
    M, N, K = 3, 70000, 65536
    A, sA = operand(rng, M, K)
    B = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda:0")
    sB = torch.rand(N, device="cuda:0")
    C = Rows(M, N, 1)
    c3gpu.c3_i8_gemm(dev(A), dev(sA), B, sB, C.ptr(), 1, M, N, K, N)
    sync()
    C.intact()
    some = np.concatenate([np.arange(40), np.arange(32760, 32790), np.arange(N - 40, N)])
    want = ref.product(A, sA, B[torch.from_numpy(some).cuda()].cpu().numpy(), sB.cpu().numpy()[some])
    np.testing.assert_array_equal(C.numpy()[:, some], want)


def experts(c3, rng, offsets, rows, E, N, K, dtype, ldc=None, shift=0):
    (A, sA), (B, sB) = operand(rng, rows, K), operand(rng, E * N, K)
    C = Rows(rows, N, dtype, ldc, shift)
    c3.c3_i8_gemm_experts(dev(A), dev(sA), dev(B), dev(sB), dev(np.asarray(offsets, np.int32)), C.ptr(), dtype, rows, E,
                          N, K, C.ld)
    sync()
    C.intact()
    want = np.full((rows, N), CANARY, np.float32)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            want[lo:hi] = ref.rounded(ref.product(A[lo:hi], sA[lo:hi], B[e * N:e * N + N], sB[e * N:e * N + N]), dtype)
    np.testing.assert_array_equal(C.numpy(), want)


EXPERTS = [(1, 1, 16, 64), (32, 32, 256, 512), (6, 4, 33, 129), (50, 8, 100, 300), (300, 3, 130, 256), (1000, 24, 200, 272),
           (700, 5, 520, 384), (900, 100, 64, 128), (2000, 70, 300, 130), (3000, 2, 300, 640), (5000, 8, 520, 512), (64, 1024, 16, 32)]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,E,N,K", EXPERTS)
def test_experts(c3gpu, rows, E, N, K, dtype):
    """Uneven experts, some without rows, rows before the first and after the last expert."""
    rng = np.random.default_rng(rows * 13 + E)
    cut = np.sort(rng.integers(0, rows + 1, E + 1)) if rows > 1 else np.array([0, 1])
    experts(c3gpu, rng, cut, rows, E, N, K, dtype, N + (5 if N % 8 else 0), 1 if N % 8 else 0)


@pytest.mark.parametrize("sizes", [[0, 0, 0, 0], [0, 0, 500, 0], [1, 0, 1, 498], [128, 256, 64, 52], [129, 255, 65, 51], [500, 0, 0, 0]])
def test_experts_loads(c3gpu, sizes):
    rng = np.random.default_rng(sum(sizes) + sizes[0])
    experts(c3gpu, rng, np.concatenate([[0], np.cumsum(sizes)]), 500, 4, 264, 256, 0)


# Shapes for every kernel that the products choose from, with stages of K that are and that are not a
# multiple of those in flight: rows of 16 and of 32 by one to eight waves, tiles of 64x32, 64x64, 128x64,
# 128x128 (a CU to itself or not) and 256x256 (by four and by eight waves, with and without tiles of up
# to 128 rows, with and without quarters in the last round); with experts, up to 64 of them and more.
EVERY = [(260, 11923, 670), (261, 10960, 540), (8572, 206, 668), (8379, 198, 545), (7432, 68, 690), (7257, 67, 555),
         (7219, 1030, 681), (8379, 912, 541), (8742, 1545, 3783), (8201, 1025, 5186), (259, 30, 670), (258, 30, 545),
         (1, 8263, 674), (1, 8222, 542), (1, 30, 669), (1, 30, 541), (17, 10708, 695), (17, 11909, 544), (130, 902, 672),
         (210, 578, 545), (6813, 65, 684), (919, 9425, 669), (18, 8413, 681), (259, 35525, 517), (390, 33214, 690),
         (271, 35512, 5192), (6716, 2060, 3971), (8410, 65, 503), (8455, 66, 690), (1, 20720, 680), (1, 20720, 501),
         (1, 8423, 797), (17, 16483, 660), (17, 17037, 3050), (17, 4176, 665), (67, 16960, 690),
         (132, 14566, 508), (68, 16577, 851), (6555, 129, 899), (75, 8259, 1038), (65, 8813, 648), (68, 8201, 863),
         (9, 8308, 500), (17, 8436, 781), (1, 30, 1823), (18, 16388, 1040), (18, 18784, 3156), (17, 4119, 4295),
         (17, 4239, 3199)]
EVERY_EXPERTS = [(2955, 100, 259, 689), (1982, 100, 321, 548), (3167, 100, 261, 676), (7214, 100, 135, 677),
                 (7332, 100, 136, 567), (4675, 100, 66, 671), (4246, 100, 65, 575), (3813, 100, 65, 683), (8938, 100, 386, 735),
                 (8915, 100, 408, 542), (8800, 24, 946, 669), (4345, 24, 1943, 568), (2521, 24, 2384, 3765),
                 (2160, 24, 2247, 4134), (7714, 70, 645, 4129), (1291, 5, 32, 717), (1327, 5, 30, 566), (101, 100, 494, 668),
                 (83, 70, 648, 540), (105, 100, 195, 691), (113, 100, 197, 548), (2216, 100, 33, 673), (2391, 100, 33, 552),
                 (1, 5, 30, 668), (1, 5, 30, 547), (1638, 100, 420, 668), (793, 70, 753, 547), (805, 70, 484, 677),
                 (904, 70, 461, 542), (1998, 100, 81, 686), (1204, 70, 131, 542), (2626, 24, 35, 691), (2508, 24, 36, 545),
                 (545, 24, 4263, 3917), (2225, 5, 7654, 3847), (812, 24, 4331, 3880), (1394, 70, 1535, 3679),
                 (3451, 100, 835, 3985), (7197, 5, 1070, 503), (627, 24, 2810, 690), (3879, 5, 4761, 559),
                 (662, 24, 2847, 506), (2318, 100, 818, 504), (2209, 100, 740, 504), (7859, 24, 65, 507),
                 (4931, 100, 67, 690), (172, 100, 81, 515), (24, 24, 337, 652), (1209, 100, 148, 508),
                 (304, 24, 653, 561), (254, 24, 265, 517), (1829, 100, 33, 656), (409, 24, 711, 652),
                 (257, 24, 2718, 542), (29, 24, 855, 501),
                 (506, 24, 1366, 506), (118, 5, 6558, 522), (886, 24, 1190, 518), (147, 5, 6517, 642),
                 (754, 24, 1251, 772), (7356, 100, 147, 503), (7269, 100, 131, 778), (1277, 24, 453, 912),
                 (908, 24, 554, 1043), (7322, 24, 98, 655), (7337, 24, 98, 823), (4821, 100, 105, 906),
                 (4639, 100, 98, 1025), (7318, 100, 66, 1178), (5517, 70, 104, 837), (57, 5, 1713, 505),
                 (7290, 24, 33, 709), (7272, 24, 34, 801), (4358, 100, 33, 507), (5620, 70, 33, 790),
                 (1, 70, 30, 770), (29, 24, 2254, 511), (26, 24, 2447, 530), (6, 5, 5093, 514), (7, 5, 1654, 1027),
                 (74, 70, 114, 908), (1, 5, 33, 1671), (6, 5, 30, 1556), (32, 70, 30, 1414), (12, 70, 31, 1552),
                 (1423, 100, 643, 508), (1040, 70, 1009, 528), (397, 24, 1355, 515), (280, 24, 664, 976),
                 (268, 24, 663, 1073), (1153, 100, 145, 905), (905, 70, 197, 1057), (413, 24, 199, 2742),
                 (192, 24, 309, 2654), (1928, 100, 34, 3044), (1112, 100, 51, 2317)]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("M,N,K", EVERY)
def test_every_kernel(c3gpu, M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    (A, sA), (B, sB) = operand(rng, M, K), operand(rng, N, K)
    C = Rows(M, N, dtype, N + N % 3, M % 2)
    c3gpu.c3_i8_gemm(dev(A), dev(sA), dev(B), dev(sB), C.ptr(), dtype, M, N, K, C.ld)
    sync()
    C.intact()
    np.testing.assert_array_equal(C.numpy(), ref.rounded(ref.product(A, sA, B, sB), dtype))


@pytest.mark.parametrize("i", range(len(EVERY_EXPERTS)))
def test_every_kernel_of_experts(c3gpu, i):
    rows, E, N, K = EVERY_EXPERTS[i]
    rng = np.random.default_rng(rows + E)
    cut = np.sort(rng.integers(0, rows + 1, E + 1))
    experts(c3gpu, rng, cut, rows, E, N, K, i % 2, N + N % 3, i % 3)


def test_experts_every_border_of_few_rows(c3gpu):
    rng = np.random.default_rng(4)
    for rows in (1, 15, 16, 17, 31, 32, 33, 47, 64, 65):
        experts(c3gpu, rng, np.array([0, rows // 2, rows // 2, rows]), rows, 3, 48, 192, 1)


@pytest.mark.parametrize("rows", [40, 600])
def test_experts_offsets_out_of_range(c3gpu, rows):
    """Offsets that are no partition: clamped to the rows that there are, nothing outside is touched."""
    import torch

    rng = np.random.default_rng(6)
    E, N, K = 6, 136, 256
    (A, sA), (B, sB) = operand(rng, rows, K), operand(rng, E * N, K)
    for offsets in ([-5, 3, 2 ** 31 - 1, 7, -2 ** 31, 9, rows + 100], [rows, 0, rows, 0, rows, 0, rows],
                    [2 ** 31 - 1] * 7, [-1] * 7):
        C = Rows(rows, N, 0)
        c3gpu.c3_i8_gemm_experts(dev(A), dev(sA), dev(B), dev(sB), dev(np.array(offsets, np.int32)), C.ptr(), 0, rows,
                                 E, N, K, N)
        sync()
        C.intact()
    torch.cuda.synchronize()


def test_unaligned_scales_and_strided_output(c3gpu):
    """Scale arrays on every 4-byte place of a 16-byte line."""
    import torch

    rng = np.random.default_rng(7)
    for M, N, K in ((40, 90, 130), (300, 520, 256)):
        (A, sA), (B, sB) = operand(rng, M, K), operand(rng, N, K)
        want = ref.rounded(ref.product(A, sA, B, sB), 0)
        for shift in (1, 2, 3):
            ta, tb = torch.full((M + 8,), np.nan, device="cuda:0"), torch.full((N + 8,), np.nan, device="cuda:0")
            ta[shift:shift + M], tb[shift:shift + N] = dev(sA), dev(sB)
            C = Rows(M, N, 0, N + shift, shift)
            c3gpu.c3_i8_gemm(dev(A), ta.data_ptr() + 4 * shift, dev(B), tb.data_ptr() + 4 * shift, C.ptr(), 0, M, N, K, C.ld)
            sync()
            C.intact()
            np.testing.assert_array_equal(C.numpy(), want)


@pytest.mark.parametrize("T", [24, 8000])
def test_in_a_captured_graph_and_on_streams(c3gpu, T):
    """Sort, product of every expert and combination in one graph, replayed on new inputs between
    eager calls; the same bits."""
    import torch

    c3 = c3gpu
    rng = np.random.default_rng(21)
    E, k, D, F = 8, 2, 520, 264
    S = T * k
    new = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda:0")  # noqa: E731
    x, w, order, offsets = new(T, D), new(T, k, t=torch.float32), new(S, t=torch.int32), new(E + 1, t=torch.int32)
    B, sB = (dev(a) for a in operand(rng, E * F, D))
    stream = torch.cuda.Stream()

    def buffers():
        return {"codes": new(S, ref.padded(D), t=torch.int8), "scales": new(S, t=torch.float32),
                "pos": new(S, t=torch.int32), "h": new(S, F), "out": new(T, F), "back": new(S, D)}

    def step(b, s):
        c3.c3_i8_dispatch(x, 0, T, D, D, order, offsets, k, E, b["codes"], b["scales"], b["pos"], s)
        c3.c3_i8_gemm_experts(b["codes"], b["scales"], B, sB, offsets, b["h"], 0, S, E, F, D, F, s)
        c3.c3_combine(b["h"], 0, T, k, F, F, b["pos"], w, b["out"], F, s)
        c3.c3_i8_dequantize(b["codes"], b["scales"], S, D, b["back"], 0, D, s)

    def fill():
        o, f, _ = routing(rng, T, E, k, 0.1)
        order.copy_(dev(o))
        offsets.copy_(dev(f))
        x.copy_(dev(rng.normal(0, 1, (T, D)).astype(np.float32)))
        w.copy_(dev(rng.random((T, k)).astype(np.float32)))

    fill()
    held = buffers()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(held, stream)
    for _ in range(4):
        fill()
        for b in held.values():
            b.fill_(0)
        graph.replay()
        eager = buffers()
        step(eager, torch.cuda.current_stream())
        sync()
        for name in held:
            assert torch.equal(held[name], eager[name]), name


def test_refusals_that_need_the_device(c3gpu):
    import torch

    c3 = c3gpu
    codes, scales = torch.zeros(8, 128, dtype=torch.int8, device="cuda:0"), torch.zeros(8, device="cuda:0")
    C = torch.zeros(8, 8, device="cuda:0")
    with pytest.raises(c3.C3Error, match="run past|overlaps"):
        c3.c3_i8_gemm(codes, scales, codes, scales, C, 1, 8, 8, 4000, 8)
    with pytest.raises(c3.C3Error, match="device memory"):
        c3.c3_i8_gemm(codes, torch.zeros(8).data_ptr(), codes, scales, C, 1, 8, 8, 128, 8)
    c3.c3_i8_gemm(codes, scales, codes, scales, C, 1, 0, 8, 128, 8)
    c3.c3_i8_gemm_experts(codes, scales, codes, scales, scales, C, 1, 8, 1, 0, 128, 8)
