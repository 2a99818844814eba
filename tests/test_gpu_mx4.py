"""MX FP4 operands and their products on the GPU against the 64-bit definitions of layer_ref:
codes, scales and values exactly; products within the bound of adding up their exact terms in
fp32 plus half a step of the output type; refusals that need the device."""
import numpy as np
import pytest

import layer_ref as ref

pytestmark = pytest.mark.gpu
HALF = {0: 2.0 ** -8, 1: 2.0 ** -24}  # half a step of bf16 and fp32, relative
INT = {0: np.int16, 1: np.int32}


def dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")


def typed(x, dtype):
    """Device tensor of float32 values in the type (bf16 values are representable already)."""
    import torch

    return dev(x).to(torch.bfloat16 if dtype == 0 else torch.float32)


def filled(shape, dtype, value=-7.0):
    import torch

    return torch.full(shape, value, dtype=torch.bfloat16 if dtype == 0 else torch.float32, device="cuda:0")


def quantise(c3, x, dtype, up=False, transpose=False, ld=None, stream=None):
    """(codes, scales) as numpy of x [rows][cols] (float32), held with row stride ld."""
    import torch

    rows, cols = x.shape
    held = np.zeros((rows, ld or cols), np.float32)
    held[:, cols:] = np.nan  # nothing past cols is read
    held[:, :cols] = x
    r, c = (cols, rows) if transpose else (rows, cols)
    nc, ns = c3.c3_mx4_bytes(r, c)
    codes = torch.full((nc + 64,), 0x5A, dtype=torch.uint8, device="cuda:0")
    scales = torch.full((ns + 64,), 0x5A, dtype=torch.uint8, device="cuda:0")
    t = typed(held, dtype)
    c3.c3_mx4_quantize(t, dtype, rows, cols, ld or cols, transpose, int(up), codes, scales, stream)
    torch.cuda.synchronize()
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    assert (codes[nc:] == 0x5A).all() and (scales[ns:] == 0x5A).all()
    return codes[:nc].reshape(r, -1), scales[:ns].reshape(r, -1)


def wide(rng, shape):
    """bf16 values over the whole exponent range, zeros and subnormals among them."""
    x = rng.normal(0, 1, shape) * np.exp2(rng.integers(-140, 128, (shape[0], 1)).astype(float))
    x *= np.exp2(rng.integers(-6, 1, shape).astype(float))
    x[rng.random(shape) < 0.05] = 0.0
    x[rng.random(shape) < 0.02] = -0.0
    return ref.bf16_round(np.clip(x, -3e38, 3e38).astype(np.float32))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 255), (7, 256), (4, 257), (1, 16384),
                                       (130, 1000), (257, 4097)])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantise(c3gpu, rows, cols, dtype, up, transpose):
    x = wide(np.random.default_rng(rows * 7919 + cols), (rows, cols))
    codes, scales = quantise(c3gpu, x, dtype, up, transpose, ld=cols + (cols % 3))
    want = ref.quantize(x.T if transpose else x, up)
    np.testing.assert_array_equal(scales, want[1])
    np.testing.assert_array_equal(codes, want[0])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,cols,ld", [(4097, 8190, 8192), (4100, 8193, 8196), (4096, 8192, 8193)])
def test_quantise_large_transposed(c3gpu, rows, cols, ld, dtype):
    """Sizes that take eight bytes of columns a lane, with ragged ends, and a stride that does not."""
    import torch

    rng = np.random.default_rng(rows + ld)
    x = ref.bf16_round(rng.normal(0, 1, (rows, cols)).astype(np.float32))
    codes, scales = quantise(c3gpu, x, dtype, False, True, ld)
    some = np.concatenate([np.arange(300), np.arange(cols - 300, cols), rng.integers(0, cols, 200)])
    want = ref.quantize(np.ascontiguousarray(x.T[some]))
    np.testing.assert_array_equal(scales[some], want[1])
    np.testing.assert_array_equal(codes[some], want[0])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantise_every_rounding_border(c3gpu, dtype, transpose):
    """Every bf16 mantissa at each distance below the block's largest, for exponents over the
    whole range (a border of e2m1 has at most two mantissa bits), the neighbours of every border in
    fp32, infinities, NaN and all-zero blocks."""
    rows = []
    mant = (1 + np.arange(128) / 128.0)
    for e in (-133, -130, -127, -126, -125, -124, -2, 0, 1, 60, 126):
        for big in (1.0, 1.5, 1.9921875):
            small = np.concatenate([mant * 2.0 ** -k for k in range(0, 6)])
            if dtype == 1:
                borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) / 4
                f = borders.astype(np.float32)
                small = np.concatenate([small, f, np.nextafter(f, np.float32(0)), np.nextafter(f, np.float32(9))])
            small = small[small <= big]
            small = np.concatenate([small, -small])
            small = np.resize(small, -(-len(small) // 31) * 31).reshape(-1, 31)
            b = np.concatenate([np.full((len(small), 1), big), small], 1) * 2.0 ** e
            rows.append(b.reshape(-1, 32))
    x = np.concatenate(rows).astype(np.float32)
    extra = np.zeros((6, 32), np.float32)
    extra[1] = -0.0
    extra[2, 5], extra[3, 31], extra[4, 0] = np.nan, np.inf, -np.inf
    extra[5] = np.float32(1e-45)
    x = np.concatenate([x, extra])
    if dtype == 0:
        x = np.where(np.isfinite(x), ref.bf16_round(x), x)
    x = x.reshape(-1, 32)
    for up in (False, True):
        want = ref.quantize(x, up)
        codes, scales = quantise(c3gpu, x.T.copy() if transpose else x, dtype, up, transpose)
        np.testing.assert_array_equal(scales, want[1])
        np.testing.assert_array_equal(codes, want[0])


def test_quantise_unaligned_input(c3gpu):
    """x on every 2-byte offset of a 16-byte line."""
    import torch

    rng = np.random.default_rng(5)
    x = ref.bf16_round(rng.normal(0, 1, (9, 520)).astype(np.float32))
    want = ref.quantize(x)
    whole = torch.zeros(9 * 520 + 8, dtype=torch.bfloat16, device="cuda:0")
    for shift in range(1, 8):
        whole[shift:shift + x.size] = typed(x.reshape(-1), 0)
        nc, ns = c3gpu.c3_mx4_bytes(9, 520)
        codes = torch.zeros(nc, dtype=torch.uint8, device="cuda:0")
        scales = torch.zeros(ns, dtype=torch.uint8, device="cuda:0")
        c3gpu.c3_mx4_quantize(whole.data_ptr() + 2 * shift, 0, 9, 520, 520, False, 0, codes, scales)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(codes.cpu().numpy().reshape(9, -1), want[0])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,cols,ld", [(1, 1, 1), (3, 33, 40), (5, 512, 512), (130, 999, 1001), (64, 4096, 4096)])
def test_dequantise(c3gpu, rows, cols, ld, dtype):
    """Every code under every scale byte, values exact; nothing past cols is written."""
    import torch

    rng = np.random.default_rng(rows + cols)
    P = ref.padded(cols)
    codes = rng.integers(0, 256, (rows, P // 2), dtype=np.uint8)
    scales = rng.integers(0, 256, (rows, P // 32), dtype=np.uint8)
    scales.reshape(-1)[:4] = (0, 1, 254, 255)
    y = filled((rows, ld), dtype)
    c3gpu.c3_mx4_dequantize(dev(codes), dev(scales), rows, cols, y, dtype, ld)
    torch.cuda.synchronize()
    got = y.float().cpu().numpy()
    with np.errstate(over="ignore"):
        want = ref.values(codes, scales, cols).astype(np.float32)
    np.testing.assert_array_equal(got[:, :cols], want)
    assert (got[:, cols:] == -7.0).all()


def operand(rng, rows, cols, scale=1.0, low=None):
    """A random operand and its values; with `low` the scale bytes are spread over a range."""
    codes, scales = ref.quantize((scale * rng.normal(0, 1, (rows, cols))).astype(np.float32))
    if low is not None:
        live = np.arange(scales.shape[1]) * 32 < cols
        scales[:, live] = rng.integers(low, low + 8, (rows, live.sum()), dtype=np.uint8)
    return codes, scales, ref.values(codes, scales, cols)


def close(got, want, bound, dtype, extra=0.0):
    """|got - want| within the sum's bound and half a step of the output's rounding."""
    limit = bound + (HALF[dtype] + extra) * (np.abs(want) + bound) + 2.0 ** -133
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 520, 16384), (2, 33, 257), (5, 100, 31), (16, 4096, 512), (17, 1030, 1000),
          (31, 65, 4100), (33, 256, 300), (64, 2050, 768), (65, 300, 5000), (100, 1, 2048), (127, 129, 640),
          (128, 128, 256), (130, 1000, 1300), (200, 3001, 600), (256, 256, 2304), (300, 520, 130),
          (513, 777, 1111), (777, 1290, 516), (1024, 2048, 512), (2100, 2309, 1030)]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(c3gpu, M, N, K, dtype):
    import torch

    rng = np.random.default_rng(M * 31 + N * 17 + K)
    a, sa, A = operand(rng, M, K)
    b, sb, B = operand(rng, N, K, 0.02, low=110)
    ldc = N + (M % 5)
    C = filled((M + 1, ldc), dtype)
    c3gpu.c3_mx4_gemm(dev(a), dev(sa), dev(b), dev(sb), C, dtype, M, N, K, ldc)
    torch.cuda.synchronize()
    got = C.double().cpu().numpy()
    close(got[:M, :N], *ref.product(A, B), dtype)
    assert (got[M:] == -7.0).all() and (got[:, N:] == -7.0).all()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("M,N,K", [(2049, 4100, 8200), (2300, 4097, 7700), (1500, 4200, 600), (40, 33000, 900)])
def test_product_large(c3gpu, M, N, K, dtype):
    """Sizes past one round of tiles of 256 and of 128, and rows that share a tile with none."""
    test_product(c3gpu, M, N, K, dtype)


@pytest.mark.parametrize("K", [512, 700, 1000, 1025, 1300, 2000, 2300])
def test_product_lengths_of_k(c3gpu, K):
    """Every remainder of the stages of 256 columns, at a size with a tile for about half the CUs."""
    test_product(c3gpu, 400, 4200, K, 0)


@pytest.mark.parametrize("M,N,K", [(700, 2000, 128), (301, 4001, 256), (2500, 5003, 200), (129, 9000, 1)])
def test_product_short_rows(c3gpu, M, N, K):
    """K within one unit of 256 columns, in tiles of 128: one for half the CUs, and two to a CU."""
    test_product(c3gpu, M, N, K, 0)


@pytest.mark.parametrize("M,N,K", [(3, 70, 600), (100, 300, 1500), (520, 700, 700), (2050, 2300, 520)])
def test_product_integers_exact_and_repeatable(c3gpu, M, N, K):
    """Small integer values: every partial sum is exact in fp32, so the product is too; and the
    same bits on a second call and on another stream."""
    import torch

    rng = np.random.default_rng(M)
    x = rng.integers(-4, 5, (M, K)).astype(np.float32)
    w = rng.integers(-4, 5, (N, K)).astype(np.float32)
    x[:, ::32], w[:, ::32] = 4, -4  # unit scale in every block
    a, sa = (dev(v) for v in ref.quantize(x))
    b, sb = (dev(v) for v in ref.quantize(w))
    out = [filled((M, N), 1) for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c3gpu.c3_mx4_gemm(a, sa, b, sb, out[0], 1, M, N, K, N)
    c3gpu.c3_mx4_gemm(a, sa, b, sb, out[1], 1, M, N, K, N)
    c3gpu.c3_mx4_gemm(a, sa, b, sb, out[2], 1, M, N, K, N, side)
    torch.cuda.synchronize()
    want = x.astype(np.int64) @ w.astype(np.int64).T
    for o in out:
        np.testing.assert_array_equal(o.cpu().numpy(), want)


@pytest.mark.parametrize("M,N,K", [(2, 40, 300), (140, 200, 700), (700, 900, 600)])
def test_product_nan_and_extreme_scales(c3gpu, M, N, K):
    """A NaN block spoils its row (or column) of C and nothing else; the smallest and largest
    scales reach infinity, zero and subnormals as fp32 does."""
    import torch

    rng = np.random.default_rng(K)
    a, sa, _ = operand(rng, M, K)
    b, sb, _ = operand(rng, N, K)
    sa[:], sb[:] = 127, 127
    sa[1, 2], sb[7, 1] = 255, 255
    C = filled((M, N), 1)
    c3gpu.c3_mx4_gemm(dev(a), dev(sa), dev(b), dev(sb), C, 1, M, N, K, N)
    torch.cuda.synchronize()
    got = C.cpu().numpy()
    nan = np.zeros((M, N), bool)
    nan[1], nan[:, 7] = True, True
    np.testing.assert_array_equal(np.isnan(got), nan)
    for ea, eb in ((0, 127), (254, 100), (10, 120)):  # 2^-127, 2^127 * 2^-27, 2^-124
        sa[:], sb[:] = ea, eb
        A, B = ref.values(a, sa, K), ref.values(b, sb, K)
        c3gpu.c3_mx4_gemm(dev(a), dev(sa), dev(b), dev(sb), C, 1, M, N, K, N)
        torch.cuda.synchronize()
        want, bound = ref.product(A, B)
        # a matrix instruction may flush terms and sums below the smallest normal
        close(C.double().cpu().numpy(), want, bound + K * 2.0 ** -126, 1)


def test_product_refuses_short_buffers(c3gpu):
    import torch

    z = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda:0")  # noqa: E731
    C = filled((4, 4), 1)
    big = 1 << 21  # a claim of 1 TiB: past A's allocation, and over whatever lies behind it
    with pytest.raises(c3gpu.C3Error) as e:
        c3gpu.c3_mx4_gemm(z(128), z(16), z(128), z(16), C, 1, big, 4, 1 << 20, 4)
    assert e.value.status in (c3gpu.C3_E_INVALID, c3gpu.C3_E_OVERLAP)
    host = np.zeros(4096, np.uint8)
    with pytest.raises(c3gpu.C3Error):
        c3gpu.c3_mx4_gemm(host.ctypes.data // 16 * 16 + 16, z(16), z(128), z(16), C, 1, 1, 1, 64, 4)
    c3gpu.c3_mx4_gemm(None, None, None, None, None, 1, 0, 4, 64, 4)  # no rows: nothing is read
    c3gpu.c3_mx4_quantize(None, 0, 0, 64, 64, False, 0, None, None)


def plan_of(rng, T, E, k, skew, absent):
    z = rng.normal(0, 1, (T, E)) + skew * rng.normal(0, 1, E)
    idx = np.argsort(-z, 1)[:, :k].astype(np.int32)
    idx[rng.random(T) < absent] = -1
    return idx, *ref.plan(idx, E)


def experts_want(A, B, idx, order, offsets, w, a_rows):
    T, k = idx.shape
    E, N, _ = B.shape
    want, bound = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        s = order[offsets[e]:offsets[e + 1]]
        if len(s):
            p, b = ref.product(A[s % T if a_rows == T else s], B[e])
            f = 1.0 if w is None else w.astype(np.float64)[s % T, s // T][:, None]
            want[s], bound[s] = p * f, b * np.abs(f)
    return want, bound


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,E,k,N,K,skew,absent,per_slot,weighted", [
    (1, 1, 1, 1, 1, 0, 0, False, True), (1, 8, 2, 100, 600, 0, 0, False, True),
    (8, 32, 4, 260, 512, 0.5, 0, False, True), (8, 32, 4, 70, 300, 0.5, 0.3, True, False),
    (3, 5, 5, 33, 257, 0, 1.0, False, True), (100, 70, 3, 129, 256, 1.0, 0.1, False, True),
    (301, 24, 3, 200, 700, 2.0, 0.1, False, True), (301, 24, 3, 200, 700, 2.0, 0.1, True, True),
    (700, 4, 2, 520, 513, 1.0, 0.0, False, True), (2050, 3, 1, 300, 300, 0.3, 0.05, False, False),
    (40, 1000, 8, 17, 64, 0.5, 0.0, False, True)])
def test_experts(c3gpu, T, E, k, N, K, skew, absent, per_slot, weighted, dtype):
    import torch

    rng = np.random.default_rng(T * 13 + E * 7 + N)
    idx, order, offsets = plan_of(rng, T, E, k, skew, absent)
    a_rows = T * k if per_slot else T
    a, sa, A = operand(rng, a_rows, K)
    b, sb, B = operand(rng, E * N, K, 0.02)
    w = rng.random((T, k)).astype(np.float32) if weighted else None
    ldc = N + (T % 3)
    C = filled((T * k + 1, ldc), dtype)
    c3gpu.c3_mx4_gemm_experts(dev(a), dev(sa), a_rows, dev(b), dev(sb), dev(order), dev(offsets),
                              None if w is None else dev(w), C, dtype, T, k, E, N, K, ldc)
    torch.cuda.synchronize()
    got = C.double().cpu().numpy()
    want, bound = experts_want(A, B.reshape(E, N, K), idx, order, offsets, w, a_rows)
    close(got[:-1, :N], want, bound, dtype, extra=2.0 ** -23)  # the weight's product rounds in fp32
    assert (got[-1] == -7.0).all() and (got[:, N:] == -7.0).all()
    absent_slots = order[offsets[E]:]
    assert (got[absent_slots, :N] == 0).all()


@pytest.mark.parametrize("per_slot", [False, True])
def test_experts_large(c3gpu, per_slot):
    test_experts(c3gpu, 4100, 3, 1, 2100, 6000, 0.3, 0.02, per_slot, True, 0)


def test_experts_short_rows(c3gpu):
    test_experts(c3gpu, 1000, 16, 2, 2001, 256, 0.5, 0.05, False, True, 1)


def test_experts_never_follow_bad_plans(c3gpu):
    """Offsets and slots outside their ranges are skipped: nothing outside C is written, and the
    slots that are in range come out right where their expert's range is."""
    import torch

    rng = np.random.default_rng(9)
    T, E, k, N, K = 50, 6, 2, 96, 256
    idx, order, offsets = plan_of(rng, T, E, k, 0.5, 0.0)
    a, sa, A = operand(rng, T, K)
    b, sb, B = operand(rng, E * N, K)
    bad = order.copy()
    bad[::7] = 1 << 30
    bad[3::7] = -5
    want, bound = experts_want(A, B.reshape(E, N, K), idx, order, offsets, None, T)
    good = np.ones(T * k, bool)
    good[order[::7]] = good[order[3::7]] = False
    for off in (offsets, np.concatenate([[-100], offsets[1:-1], [1 << 30]]).astype(np.int32)):
        C = filled((T * k + 1, N), 1)
        c3gpu.c3_mx4_gemm_experts(dev(a), dev(sa), T, dev(b), dev(sb), dev(bad), dev(off), None, C, 1, T, k, E, N,
                                  K, N)
        torch.cuda.synchronize()
        got = C.double().cpu().numpy()
        close(got[:-1][good], want[good], bound[good], 1)
        assert (got[:-1][~good] == -7.0).all() and (got[-1] == -7.0).all()
    C = filled((T * k + 1, N), 1)
    falling = offsets[::-1].copy()
    c3gpu.c3_mx4_gemm_experts(dev(a), dev(sa), T, dev(b), dev(sb), dev(order), dev(falling), None, C, 1, T, k, E, N,
                              K, N)
    torch.cuda.synchronize()
    assert (C[-1] == -7.0).all().item()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("cols", [1, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("rows", [2, 513, 1500])
def test_dequantise_narrow(c3gpu, rows, cols, dtype):
    """Few columns and many rows: one lane or a few hold a row, over several workgroups."""
    test_dequantise(c3gpu, rows, cols, cols + 3, dtype)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("tokens", range(1, 10))
def test_quantise_transposed_read_back(c3gpu, tokens, dtype):
    """A few tokens quantised along the tokens: the operand's rows are the features, its columns few."""
    import torch

    features = 700
    x = wide(np.random.default_rng(tokens), (tokens, features))
    codes, scales = quantise(c3gpu, x, dtype, False, True)
    y = filled((features + 1, tokens), 1)
    c3gpu.c3_mx4_dequantize(dev(codes), dev(scales), features, tokens, y, 1, tokens)
    torch.cuda.synchronize()
    want = ref.values(*ref.quantize(np.ascontiguousarray(x.T)), tokens).astype(np.float32)
    np.testing.assert_array_equal(y[:features].cpu().numpy(), want)
    assert (y[features] == -7.0).all().item()


def test_experts_wide(c3gpu):
    """More workgroups than 2^22: 64 experts' rows of 1.4 million columns, on columns spread over them."""
    import torch

    rng = np.random.default_rng(12)
    T, E, k, N, K = 64, 64, 8, 1_400_000, 256
    idx, order, offsets = plan_of(rng, T, E, k, 0.0, 0.0)
    a, sa, A = operand(rng, T, K)
    b = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda:0")
    sb = torch.randint(118, 124, (E, N, K // 32), dtype=torch.uint8, device="cuda:0")
    C = filled((T * k, N), 0, float("nan"))
    c3gpu.c3_mx4_gemm_experts(dev(a), dev(sa), T, b, sb, dev(order), dev(offsets), None, C, 0, T, k, E, N, K, N)
    torch.cuda.synchronize()
    assert not C.isnan().any().item()
    some = dev(np.concatenate([np.arange(40), rng.integers(0, N, 200), np.arange(N - 40, N)]))
    B = ref.values(b[:, some].cpu().numpy(), sb[:, some].cpu().numpy(), K)
    want, bound = experts_want(A, B, idx, order, offsets, None, T)
    close(C[:, some].double().cpu().numpy(), want, bound, 0)
    del b, sb, C
    torch.cuda.empty_cache()


def test_quantise_more_rows_than_a_launch_takes(c3gpu):
    """2^28 rows and some of one value each, which repeat 257 others."""
    import torch

    rng = np.random.default_rng(8)
    n, rows = 257, (1 << 28) + 19
    x = wide(rng, (n, 1))
    want = ref.quantize(x)
    t = typed(x, 0).repeat(rows // n + 1, 1)[:rows].contiguous()
    nc, ns = c3gpu.c3_mx4_bytes(rows, 1)
    codes = torch.full((nc + 64,), 0x5A, dtype=torch.uint8, device="cuda:0")
    scales = torch.full((ns + 64,), 0x5A, dtype=torch.uint8, device="cuda:0")
    c3gpu.c3_mx4_quantize(t, 0, rows, 1, 1, False, 0, codes, scales)
    torch.cuda.synchronize()
    assert (codes[nc:] == 0x5A).all().item() and (scales[ns:] == 0x5A).all().item()
    step = n * 4096
    for got, one in ((codes[:nc].view(rows, -1), want[0]), (scales[:ns].view(rows, -1), want[1])):
        all_of = dev(one).repeat(4096, 1)
        for r in range(0, rows, step):
            part = got[r:r + step]
            assert torch.equal(part, all_of[:len(part)]), r
    del t, codes, scales, got, part
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,E,k,N,K,skew,absent", [
    (3000, 64, 6, 520, 300, 0.5, 0.05), (1500, 70, 6, 140, 513, 1.5, 0.0), (1500, 70, 6, 700, 513, 0.5, 0.0),
    (4000, 256, 8, 200, 300, 0.5, 0.1), (6000, 600, 16, 65, 300, 1.0, 0.02), (1500, 130, 8, 500, 300, 0.5, 0.02)])
def test_experts_many_in_tiles(c3gpu, T, E, k, N, K, skew, absent, dtype):
    """64 experts and more, with rows enough for the tile kernels."""
    test_experts(c3gpu, T, E, k, N, K, skew, absent, False, True, dtype)


@pytest.mark.parametrize("M,N,K", [(32, 1100, 16384), (20, 1000, 8200), (17, 520, 30000)])
def test_product_few_rows_long_k(c3gpu, M, N, K):
    """Up to sixteen waves a workgroup, which split K among them."""
    test_product(c3gpu, M, N, K, 0)


@pytest.mark.parametrize("T,E,k,N,K", [(40, 4, 2, 600, 9000), (100, 8, 2, 260, 8500), (6, 3, 2, 500, 20000)])
def test_experts_few_rows_long_k(c3gpu, T, E, k, N, K):
    test_experts(c3gpu, T, E, k, N, K, 0.3, 0.05, True, True, 1)
