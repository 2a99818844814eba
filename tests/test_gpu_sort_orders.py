"""Sorting by orders that are no plan: entries that are no slot, slots that are missing (with a place
left in pos from an earlier sort) and slots named more than once. The rows are the same whatever the
size of the batch, on both sides of the one from which tokens and not rows are gone through."""
import numpy as np
import pytest

import sort_ref as ref
from test_gpu_i8 import wide
from test_gpu_sort import CANARY, Rows, dev, routing, sync, values

pytestmark = pytest.mark.gpu

E = 64
KINDS = ["dropped", "twice", "one slot", "both", "behind the end"]


def order_of(rng, T, k, kind):
    """(order, offsets, n)."""
    order, offsets, n = routing(rng, T, E, k, 0.05)
    S = T * k
    if kind in ("dropped", "both"):
        order = np.where(rng.random(S) < 0.2, rng.choice([-1, S, 2 ** 31 - 1, -2 ** 31, S + 5], S), order)
    if kind in ("twice", "both"):
        order = np.where(rng.random(S) < 0.1, order[rng.permutation(S)], order)
    if kind == "one slot":
        order[S // 4:S // 4 + 200] = S - 1
    if kind == "behind the end":  # slots named on both sides of the last row that counts
        n = S // 2
        order[n - 3:n + 3] = order[n]
        offsets[-1] = n
    return order.astype(np.int32), offsets, n


def check_pos(got, old, order, n):
    """Slots not named keep their place; the others have one of those that name them."""
    S = len(old)
    named = np.zeros(S, bool)
    fits = np.zeros(S, bool)
    p = np.flatnonzero((order >= 0) & (order < S))
    named[order[p]] = True
    value = np.where(p < n, p, -1)
    fits[order[p][got[order[p]] == value]] = True
    np.testing.assert_array_equal(got[~named], old[~named])
    assert fits[named].all()


def rows_written(order, n):
    S = len(order)
    return (np.arange(S) < n) & (order >= 0) & (order < S)


# T, k, cols: the first of each list are below the size from which tokens are gone through, the others above
SORTS = [(40, 3, 72, 0), (40, 3, 72, 1), (5000, 4, 1032, 0), (2500, 6, 1101, 0), (4000, 4, 600, 1), (9000, 5, 257, 1),
         (1700, 4, 3001, 0), (700, 8, 3001, 0), (90000, 8, 24, 0), (9000, 1, 8000, 0), (300000, 8, 8, 0), (1100000, 3, 4, 1),
         (700, 40, 520, 0), (320, 37, 2400, 0)]
QUANTISED = [(40, 3, 300, 0), (40, 3, 300, 1), (10000, 7, 100, 0), (5000, 3, 1032, 0), (1500, 2, 5000, 1), (300, 3, 17000, 0),
             (9000, 5, 200, 1), (2000, 40, 100, 0), (400, 17, 1100, 1)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,k,cols,dtype", SORTS)
def test_dispatch(c3gpu, T, k, cols, dtype, kind):
    rng = np.random.default_rng(T + cols)
    S = T * k
    if kind == "one slot" and S < 400:
        T, S = T * 4, S * 4
    order, offsets, n = order_of(rng, T, k, kind)
    old = rng.permutation(S).astype(np.int32)
    x, y, pos = Rows(T, cols, dtype, values=values(rng, (T, cols), dtype)), Rows(S, cols, dtype, cols + 3), dev(old)
    c3gpu.c3_dispatch(x.ptr(), dtype, T, cols, cols, dev(order), dev(offsets), k, E, y.ptr(), y.ld, pos)
    sync()
    y.intact()
    here, got = rows_written(order, n), y.numpy()
    np.testing.assert_array_equal(got[here], x.numpy()[order[here] % T])
    assert (got[~here] == CANARY).all()
    check_pos(pos.cpu().numpy(), old, order, n)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,k,cols,dtype", QUANTISED)
def test_sorted_quantise(c3gpu, T, k, cols, dtype, kind):
    import torch

    rng = np.random.default_rng(T + cols)
    S = T * k
    if kind == "one slot" and S < 400:
        T, S = T * 4, S * 4
    order, offsets, n = order_of(rng, T, k, kind)
    old = rng.permutation(S).astype(np.int32)
    x = wide(rng, T, cols, dtype)
    X, P, pos = Rows(T, cols, dtype, values=x), ref.padded(cols), dev(old)
    codes = torch.full((S + 1, P), 0x5A, dtype=torch.int8, device="cuda:0")
    scales = torch.full((S + 1,), CANARY, device="cuda:0")
    c3gpu.c3_i8_dispatch(X.ptr(), dtype, T, cols, cols, dev(order), dev(offsets), k, E, codes, scales, pos)
    sync()
    here, want = rows_written(order, n), ref.quantize(x)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    np.testing.assert_array_equal(codes[:S][here], want[0][order[here] % T])
    np.testing.assert_array_equal(scales[:S][here], want[1][order[here] % T])
    assert (codes[S] == 0x5A).all() and scales[S] == CANARY
    assert (codes[:S][~here] == 0x5A).all() and (scales[:S][~here] == CANARY).all()
    check_pos(pos.cpu().numpy(), old, order, n)


@pytest.mark.parametrize("last", [-5, 0, 7, 1 << 30])
def test_offsets_out_of_range_in_large_batches(c3gpu, last):
    import torch

    rng = np.random.default_rng(3)
    T, k, cols = 5000, 4, 1032
    S, P = T * k, ref.padded(cols)
    order, offsets, _ = order_of(rng, T, k, "both")
    offsets[-1] = last
    n, old = min(max(last, 0), S), rng.permutation(S).astype(np.int32)
    x = values(rng, (T, cols), 0)
    X, y, pos, here = Rows(T, cols, 0, values=x), Rows(S, cols, 0), dev(old), rows_written(order, n)
    c3gpu.c3_dispatch(X.ptr(), 0, T, cols, cols, dev(order), dev(offsets), k, E, y.ptr(), cols, pos)
    sync()
    got = y.numpy()
    np.testing.assert_array_equal(got[here], x[order[here] % T])
    assert (got[~here] == CANARY).all()
    check_pos(pos.cpu().numpy(), old, order, n)
    codes, pos = torch.full((S, P), 0x5A, dtype=torch.int8, device="cuda:0"), dev(old)
    scales = torch.full((S,), CANARY, device="cuda:0")
    c3gpu.c3_i8_dispatch(X.ptr(), 0, T, cols, cols, dev(order), dev(offsets), k, E, codes, scales, pos)
    sync()
    want, got = ref.quantize(x), codes.cpu().numpy()
    np.testing.assert_array_equal(got[here], want[0][order[here] % T])
    assert (got[~here] == 0x5A).all() and (scales.cpu().numpy()[~here] == CANARY).all()
    check_pos(pos.cpu().numpy(), old, order, n)


def test_large_batches_in_a_captured_graph(c3gpu):
    """A step whose dropped choices change from replay to replay, its pos and rows kept: rows that no
    choice has stay as they were, also where pos names them from the replay before."""
    import torch

    rng = np.random.default_rng(5)
    T, k, cols = 5000, 3, 1032
    S = T * k
    x, y = dev(values(rng, (T, cols), 1)), torch.zeros(S, cols, device="cuda:0")
    order, offsets = torch.zeros(S, dtype=torch.int32, device="cuda:0"), torch.zeros(E + 1, dtype=torch.int32, device="cuda:0")
    pos = torch.full((S,), -1, dtype=torch.int32, device="cuda:0")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c3gpu.c3_dispatch(x, 1, T, cols, cols, order, offsets, k, E, y, cols, pos, stream)
    for kind in ("dropped", "both", "twice", "dropped"):
        o, f, n = order_of(rng, T, k, kind)
        order.copy_(dev(o))
        offsets.copy_(dev(f))
        x.copy_(dev(values(rng, (T, cols), 1)))
        y.fill_(CANARY)
        old = pos.cpu().numpy()
        graph.replay()
        sync()
        here, got = rows_written(o, n), y.cpu().numpy()
        np.testing.assert_array_equal(got[here], x.cpu().numpy()[o[here] % T])
        assert (got[~here] == CANARY).all()
        check_pos(pos.cpu().numpy(), old, o, n)


def test_rows_past_32_bits_by_token(c3gpu):
    """Large batches whose rows lie past 2^31 elements and 2^32 bytes."""
    import torch

    rng = np.random.default_rng(6)
    T, k, cols, ld = 2100, 4, 3000, 1 << 20
    S = T * k
    order, offsets, n = order_of(rng, T, k, "twice")
    x = values(rng, (T, cols), 0)
    y = torch.zeros(S * ld, dtype=torch.bfloat16, device="cuda:0")
    X, pos, here = Rows(T, cols, 0, values=x), dev(rng.permutation(S).astype(np.int32)), rows_written(order, n)
    c3gpu.c3_dispatch(X.ptr(), 0, T, cols, cols, dev(order), dev(offsets), k, E, y, ld, pos)
    sync()
    got = y.view(S, ld)[:, :cols].float().cpu().numpy()
    np.testing.assert_array_equal(got[here], x[order[here] % T])
    assert not got[~here].any() and not bool(y.view(S, ld)[:, cols:cols + 64].any())


def test_codes_past_32_bits_by_token(c3gpu):
    import torch

    g = torch.Generator(device="cuda:0").manual_seed(1)
    rng = np.random.default_rng(7)
    T, k, cols = 34000, 8, 16384
    S = T * k
    order, offsets, n = order_of(rng, T, k, "twice")
    x = torch.randn(T, cols, generator=g, device="cuda:0").bfloat16()
    A, sA = torch.empty(T, cols, dtype=torch.int8, device="cuda:0"), torch.empty(T, device="cuda:0")
    c3gpu.c3_i8_quantize(x, 0, T, cols, cols, A, sA)
    codes, scales = torch.full((S, cols), 0x5A, dtype=torch.int8, device="cuda:0"), torch.zeros(S, device="cuda:0")
    c3gpu.c3_i8_dispatch(x, 0, T, cols, cols, dev(order), dev(offsets), k, E, codes, scales,
                         dev(rng.permutation(S).astype(np.int32)))
    sync()
    here = rows_written(order, n)
    for p in np.array_split(np.flatnonzero(here), 16):
        t, at = dev(order[p] % T).long(), dev(p)
        assert torch.equal(codes[at], A[t]) and torch.equal(scales[at], sA[t])
    assert bool((codes[dev(np.flatnonzero(~here))] == 0x5A).all())
