"""Rows sorted by expert and back on the GPU against the definitions of sort_ref: sorted rows and
positions exactly, sums and gradients within bounds counted from their roundings."""
import numpy as np
import pytest

import sort_ref as ref

pytestmark = pytest.mark.gpu
CANARY = -7.0


def dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")


def sync():
    import torch

    torch.cuda.synchronize()


class Rows:
    """A matrix of the type on the device: row stride ld, its first element `shift` elements past a
    16-byte line, everything around it a canary."""

    def __init__(self, rows, cols, dtype, ld=None, shift=0, values=None):
        import torch

        self.rows, self.cols, self.ld, self.shift, self.dtype = rows, cols, ld or cols, shift, dtype
        kind = torch.bfloat16 if dtype == 0 else torch.float32
        self.whole = torch.full((shift + rows * self.ld + 16,), CANARY, dtype=kind, device="cuda:0")
        if values is not None:
            self.view()[:] = dev(values.astype(np.float32)).to(kind)

    def view(self):
        return self.whole[self.shift:self.shift + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols]

    def ptr(self):
        return self.whole.data_ptr() + self.shift * self.whole.element_size()

    def numpy(self):
        return self.view().float().cpu().numpy()

    def intact(self):
        """Nothing around the matrix was written."""
        w = self.whole.clone()
        w[self.shift:self.shift + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = CANARY
        assert bool((w == CANARY).all())


def routing(rng, T, E, k, masked):
    """(order, offsets, n) of random distinct choices, some tokens and choices without."""
    idx = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    idx[rng.random(T) < masked] = -1
    idx[rng.random((T, k)) < masked / 2] = E + 3
    order, offsets = ref.plan(idx, E)
    return order, offsets, int(offsets[-1])


def values(rng, shape, dtype):
    x = rng.normal(0, 1, shape).astype(np.float32)
    return ref.bf16_round(x) if dtype == 0 else x


# T, E, k, cols, row stride past cols, elements past a 16-byte line, share of tokens without experts
CASES = [(1, 1, 1, 1, 0, 0, 0.0), (1, 4, 4, 4096, 0, 0, 0.0), (1, 8, 3, 16385, 7, 1, 0.0), (3, 8, 2, 7, 1, 3, 0.0),
         (8, 32, 4, 4096, 0, 0, 0.0), (17, 5, 3, 129, 0, 1, 0.3), (33, 6, 2, 1000, 24, 0, 0.1),
         (5, 64, 64, 40, 0, 0, 0.2), (700, 16, 8, 520, 0, 0, 0.1), (6000, 64, 7, 65, 3, 5, 0.05),
         (9000, 256, 8, 8, 0, 0, 0.0), (4099, 24, 3, 2049, 0, 0, 0.1), (40, 8, 2, 640, 0, 0, 1.0),
         (300, 8, 2, 5001, 0, 0, 0.1)]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,E,k,cols,more,shift,masked", CASES)
def test_dispatch(c3gpu, T, E, k, cols, more, shift, masked, dtype):
    import torch

    rng = np.random.default_rng(T * 131 + cols)
    order, offsets, n = routing(rng, T, E, k, masked)
    x = Rows(T, cols, dtype, cols + more, shift, values(rng, (T, cols), dtype))
    y = Rows(T * k, cols, dtype, cols + 2 * more, shift // 2)
    pos = torch.full((T * k + 8,), -9, dtype=torch.int32, device="cuda:0")
    c3gpu.c3_dispatch(x.ptr(), dtype, T, cols, x.ld, dev(order), dev(offsets), k, E, y.ptr(), y.ld, pos)
    sync()
    got = pos.cpu().numpy()
    np.testing.assert_array_equal(got[:T * k], ref.positions(order, n, T * k))
    assert (got[T * k:] == -9).all()
    y.intact()
    got = y.numpy()
    np.testing.assert_array_equal(got[:n], ref.sort_rows(x.numpy(), order, n))
    assert (got[n:] == CANARY).all()  # rows of no expert are left alone


@pytest.mark.parametrize("T,cols", [(5, 24), (4000, 136)])
def test_dispatch_copies_every_bit(c3gpu, T, cols):
    import torch

    rng = np.random.default_rng(1)
    order, offsets, n = routing(rng, T, 8, 2, 0.0)
    x = rng.integers(-32768, 32768, (T, cols)).astype(np.int16)
    y, pos = torch.zeros(2 * T, cols, dtype=torch.int16, device="cuda:0"), torch.empty(2 * T, dtype=torch.int32, device="cuda:0")
    c3gpu.c3_dispatch(dev(x), 0, T, cols, cols, dev(order), dev(offsets), 2, 8, y, cols, pos)
    sync()
    np.testing.assert_array_equal(y.cpu().numpy()[:n], ref.sort_rows(x, order, n))


@pytest.mark.parametrize("T,cols", [(9, 40), (3000, 264)])
@pytest.mark.parametrize("last", [None, -5, 1 << 30])
def test_dispatch_skips_what_is_no_slot(c3gpu, T, cols, last):
    import torch

    rng = np.random.default_rng(2)
    k, E = 3, 8
    order, offsets, n = routing(rng, T, E, k, 0.0)
    S = T * k
    bad = rng.random(S) < 0.2
    order = np.where(bad, rng.choice([-1, S, 2 ** 31 - 1, -2 ** 31, S + 5], S), order).astype(np.int32)
    if last is not None:
        offsets = offsets.copy()
        offsets[-1] = last
        n = min(max(last, 0), S)
    x, y = Rows(T, cols, 0, values=values(rng, (T, cols), 0)), Rows(S, cols, 0)
    pos = torch.full((S,), -2, dtype=torch.int32, device="cuda:0")
    c3gpu.c3_dispatch(x.ptr(), 0, T, cols, cols, dev(order), dev(offsets), k, E, y.ptr(), cols, pos)
    sync()
    np.testing.assert_array_equal(pos.cpu().numpy(), ref.positions(order, n, S))
    got, src = y.numpy(), x.numpy()
    for p in range(S):
        if p < n and not bad[p]:
            assert (got[p] == src[order[p] % T]).all()
        else:
            assert (got[p] == CANARY).all()
    y.intact()


def plan_of(rng, T, E, k, masked):
    order, offsets, n = routing(rng, T, E, k, masked)
    return ref.positions(order, n, T * k).reshape(k, T), n


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,E,k,cols,more,shift,masked", CASES)
def test_combine(c3gpu, T, E, k, cols, more, shift, masked, weighted, dtype):
    rng = np.random.default_rng(T * 17 + cols)
    pos, n = plan_of(rng, T, E, k, masked)
    y = values(rng, (T * k, cols), dtype)
    y[n:] = np.nan  # rows without a slot are not read
    w = rng.normal(0, 1, (T, k)).astype(np.float32) if weighted else None
    if weighted:
        w.T[pos < 0] = np.nan  # neither are weights of absent choices
    Y = Rows(T * k, cols, dtype, cols + more, shift, y)
    out = Rows(T, cols, dtype, cols + 2 * more, shift // 2)
    c3gpu.c3_combine(Y.ptr(), dtype, T, k, cols, Y.ld, dev(pos), None if w is None else dev(w), out.ptr(), out.ld)
    sync()
    out.intact()
    want, bound = ref.combine(y, pos, w)
    limit = bound + ref.HALF[dtype] * (np.abs(want) + bound)
    assert (np.abs(out.numpy() - want) <= limit).all()
    assert (out.numpy()[(pos < 0).all(0)] == 0).all()


def test_combine_keeps_rows_apart_and_skips_bad_positions(c3gpu):
    rng = np.random.default_rng(6)
    T, k, cols = 50, 4, 72
    pos, n = plan_of(rng, T, 8, k, 0.0)
    y = values(rng, (T * k, cols), 0)
    w = rng.random((T, k)).astype(np.float32)
    y[pos[1, 3], 5], y[pos[0, 4], 6], y[pos[3, 5], 7] = np.nan, np.inf, -np.inf
    pos[2, 10], pos[0, 11], pos[3, 12], pos[1, 13] = T * k, -2 ** 31, 2 ** 31 - 1, -7
    Y, out = Rows(T * k, cols, 0, values=y), Rows(T, cols, 0)
    c3gpu.c3_combine(Y.ptr(), 0, T, k, cols, cols, dev(pos), dev(w), out.ptr(), cols)
    sync()
    got = out.numpy()
    assert np.isnan(got[3, 5]) and got[4, 6] == np.inf and got[5, 7] == -np.inf
    odd = ~np.isfinite(got)
    assert odd.sum() == 3
    want, bound = ref.combine(np.where(np.isfinite(y), y, 0), pos, w)
    assert (np.abs(got - want) <= bound + ref.HALF[0] * (np.abs(want) + bound))[~odd].all()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,E,k,cols,more,shift,masked", CASES)
def test_combine_backward(c3gpu, T, E, k, cols, more, shift, masked, weighted, dtype):
    import torch

    rng = np.random.default_rng(T * 19 + cols)
    pos, n = plan_of(rng, T, E, k, masked)
    y, dout = values(rng, (T * k, cols), dtype), values(rng, (T, cols), dtype)
    y[n:] = np.nan
    w = rng.normal(0, 1, (T, k)).astype(np.float32) if weighted else None
    Y, D = Rows(T * k, cols, dtype, cols + more, shift, y), Rows(T, cols, dtype, cols + 2 * more, shift // 2, dout)
    want, written, dw, bound = ref.combine_gradient(dout, y, pos, w)
    for with_dw in (True, False):
        dY = Rows(T * k, cols, dtype, cols + 3 * more, shift // 3)
        dW = torch.full((T * k + 4,), CANARY, device="cuda:0")
        c3gpu.c3_combine_backward(D.ptr(), dtype, T, k, cols, D.ld, Y.ptr() if with_dw else None, Y.ld, dev(pos),
                                  None if w is None else dev(w), dY.ptr(), dY.ld, dW if with_dw else None)
        sync()
        dY.intact()
        got = dY.numpy()
        assert (got[~written] == CANARY).all()
        # the product is rounded to fp32, then to the type
        limit = (ref.HALF[dtype] + 2.0 ** -24) * 1.01 * np.abs(want) + ref.TINY
        assert (np.abs(got - want) <= limit)[written].all()
        got = dW.cpu().numpy()
        assert (got[T * k:] == CANARY).all()
        if with_dw:
            assert (np.abs(got[:T * k].reshape(T, k) - dw) <= bound).all()
            assert (got[:T * k].reshape(T, k).T[pos < 0] == 0).all()
        else:
            assert (got == CANARY).all()


def test_combine_backward_skips_bad_positions(c3gpu):
    import torch

    rng = np.random.default_rng(8)
    T, k, cols = 60, 3, 200
    pos, n = plan_of(rng, T, 8, k, 0.0)
    pos[0, 10], pos[1, 11], pos[2, 12], pos[0, 13] = T * k, -2 ** 31, 2 ** 31 - 1, -7
    y, dout, w = values(rng, (T * k, cols), 1), values(rng, (T, cols), 1), rng.random((T, k)).astype(np.float32)
    dY, dW = Rows(T * k, cols, 1), torch.full((T, k), CANARY, device="cuda:0")
    c3gpu.c3_combine_backward(dev(dout), 1, T, k, cols, cols, dev(y), cols, dev(pos), dev(w), dY.ptr(), cols, dW)
    sync()
    want, written, dw, bound = ref.combine_gradient(dout, y, pos, w)
    dY.intact()
    assert (dY.numpy()[~written] == CANARY).all() and (~written).sum() == 4
    assert (np.abs(dY.numpy() - want) <= 2.1 * 2.0 ** -24 * np.abs(want) + ref.TINY)[written].all()
    assert (np.abs(dW.cpu().numpy() - dw) <= bound).all()


@pytest.mark.parametrize("T,k,cols,dtype", [(2500, 8, 2049, 0), (9000, 6, 2400, 0), (4000, 6, 4301, 0), (5200, 3, 4100, 1), (9000, 2, 4096, 0),
                                              (6000, 5, 2000, 1)])
def test_traffic_past_the_caches(c3gpu, T, k, cols, dtype):
    """Sizes that take other kernels: sorted token by token with few and with many choices, fewer
    choices in flight, rows by more lanes. Sums and gradients of some tokens, the sort of all."""
    import torch

    rng = np.random.default_rng(T + cols)
    g = torch.Generator(device="cuda:0").manual_seed(T)
    kind = torch.bfloat16 if dtype == 0 else torch.float32
    order, offsets, n = routing(rng, T, 16, k, 0.05)
    S = T * k
    new = lambda *s: torch.randn(*s, generator=g, device="cuda:0").to(kind)  # noqa: E731
    x, pos = new(T, cols), torch.full((S,), -9, dtype=torch.int32, device="cuda:0")
    y = torch.full((S, cols), CANARY, dtype=kind, device="cuda:0")
    c3gpu.c3_dispatch(x, dtype, T, cols, cols, dev(order), dev(offsets), k, 16, y, cols, pos)
    sync()
    want = ref.positions(order, n, S)
    np.testing.assert_array_equal(pos.cpu().numpy(), want)
    assert torch.equal(y[:n], x[dev(order[:n] % T).long()]) and bool((y[n:] == CANARY).all())

    y = new(S, cols)
    w, dout = torch.randn(T, k, generator=g, device="cuda:0"), new(T, cols)
    out, dy, dw = new(T, cols), torch.full((S, cols), CANARY, dtype=kind, device="cuda:0"), torch.empty(T, k, device="cuda:0")
    c3gpu.c3_combine(y, dtype, T, k, cols, cols, pos, w, out, cols)
    c3gpu.c3_combine_backward(dout, dtype, T, k, cols, cols, y, cols, pos, w, dy, cols, dw)
    sync()
    assert bool((dy[n:] == CANARY).all())
    some = np.concatenate([np.arange(40), rng.integers(0, T, 200), np.arange(T - 40, T)])
    at = want.reshape(k, T)[:, some]
    rows = y[dev(np.maximum(at, 0).reshape(-1)).long()].float().cpu().numpy()
    local = np.where(at >= 0, np.arange(at.size).reshape(at.shape), -1)  # the rows of these tokens alone
    take = lambda t: t[dev(some).long()].float().cpu().numpy()  # noqa: E731
    sums, bound = ref.combine(rows, local, take(w))
    assert (np.abs(take(out) - sums) <= bound + ref.HALF[dtype] * (np.abs(sums) + bound)).all()
    d, written, dws, bound = ref.combine_gradient(take(dout), rows, local, take(w))
    got = dy[dev(np.maximum(at, 0).reshape(-1)).long()].float().cpu().numpy()
    assert (np.abs(got - d) <= (ref.HALF[dtype] + 2.0 ** -24) * 1.01 * np.abs(d) + ref.TINY)[written].all()
    assert (np.abs(take(dw) - dws) <= bound).all()


def test_offsets_past_32_bits(c3gpu):
    """Rows of y whose byte and element offsets pass 2^32 and 2^31."""
    import torch

    rng = np.random.default_rng(3)
    T, k, cols, ld = 2100, 2, 40, 1 << 20
    order, offsets, n = routing(rng, T, 8, k, 0.0)
    x = values(rng, (T, cols), 0)
    y = torch.empty(T * k * ld, dtype=torch.bfloat16, device="cuda:0")
    pos = torch.empty(T * k, dtype=torch.int32, device="cuda:0")
    X = Rows(T, cols, 0, values=x)
    c3gpu.c3_dispatch(X.ptr(), 0, T, cols, cols, dev(order), dev(offsets), k, 8, y, ld, pos)
    sync()
    rows = y.view(T * k, ld)[:, :cols]
    np.testing.assert_array_equal(rows.float().cpu().numpy()[:n], ref.sort_rows(x, order, n))
    out = Rows(T, cols, 0)
    c3gpu.c3_combine(y, 0, T, k, cols, ld, pos, None, out.ptr(), cols)
    sync()
    np.testing.assert_array_equal(out.numpy(), 2 * x)
    dw = torch.empty(T, k, device="cuda:0")
    w = np.full((T, k), 0.5, np.float32)
    dy = torch.empty_like(y)
    c3gpu.c3_combine_backward(X.ptr(), 0, T, k, cols, cols, y, ld, pos, dev(w), dy, ld, dw)
    sync()
    np.testing.assert_array_equal(dy.view(T * k, ld)[:, :cols].float().cpu().numpy()[:n], 0.5 * ref.sort_rows(x, order, n))
    want = (x.astype(np.float64) ** 2).sum(1)
    assert (np.abs(dw.cpu().numpy() - want[:, None]) <= 1.01 * (cols + 16) * 2.0 ** -24 * want[:, None]).all()


@pytest.mark.parametrize("T,E,k,cols", [(4, 8, 2, 96), (2000, 16, 4, 512), (4000, 16, 8, 1024)])
def test_in_a_captured_graph(c3gpu, T, E, k, cols):
    """Dispatch, combine and its gradient captured once, replayed on new inputs with eager work of
    the same buffers' shapes between the replays; the same bits as eager calls."""
    import torch

    c3 = c3gpu
    rng = np.random.default_rng(9)
    stream = torch.cuda.Stream()
    new = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda:0")  # noqa: E731
    i32 = torch.int32
    x, w, g = new(T, cols), new(T, k, t=torch.float32), new(T, cols)
    order, offsets = new(T * k, t=i32), new(E + 1, t=i32)

    def buffers():
        return {"y": new(T * k, cols), "pos": new(T * k, t=i32), "out": new(T, cols), "dy": new(T * k, cols),
                "dw": new(T, k, t=torch.float32)}

    def step(b, s):
        c3.c3_dispatch(x, 0, T, cols, cols, order, offsets, k, E, b["y"], cols, b["pos"], s)
        c3.c3_combine(b["y"], 0, T, k, cols, cols, b["pos"], w, b["out"], cols, s)
        c3.c3_combine_backward(g, 0, T, k, cols, cols, b["y"], cols, b["pos"], w, b["dy"], cols, b["dw"], s)

    def fill():
        o, f, _ = routing(rng, T, E, k, 0.1)
        order.copy_(dev(o))
        offsets.copy_(dev(f))
        for t in (x, w, g):
            t.copy_(dev(rng.normal(0, 1, t.shape).astype(np.float32)))

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


def test_an_expert_named_twice(c3gpu):
    """Both choices of a token may have one expert: two slots, two rows, two weights."""
    import torch

    rng = np.random.default_rng(13)
    T, E, k, cols = 200, 4, 3, 70
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    order, offsets = ref.plan(idx, E)
    x, w = Rows(T, cols, 1, values=values(rng, (T, cols), 1)), rng.random((T, k)).astype(np.float32)
    y, pos = Rows(T * k, cols, 1), torch.empty(T * k, dtype=torch.int32, device="cuda:0")
    out = Rows(T, cols, 1)
    c3gpu.c3_dispatch(x.ptr(), 1, T, cols, cols, dev(order), dev(offsets), k, E, y.ptr(), cols, pos)
    c3gpu.c3_combine(y.ptr(), 1, T, k, cols, cols, pos, dev(w), out.ptr(), cols)
    sync()
    np.testing.assert_array_equal(y.numpy(), ref.sort_rows(x.numpy(), order, T * k))
    want, bound = ref.combine(y.numpy(), ref.positions(order, T * k, T * k).reshape(k, T), w)
    assert (np.abs(out.numpy() - want) <= bound + ref.HALF[1] * (np.abs(want) + bound)).all()


def test_calls_from_several_host_threads(c3gpu):
    """Threads with a stream and buffers each, all operators in turn; every one gets its own answer."""
    import threading

    import torch

    c3 = c3gpu
    T, E, k, cols, n = 300, 8, 2, 264, 4
    rng = np.random.default_rng(14)
    jobs, bad = [], []
    for _ in range(n):
        order, offsets, m = routing(rng, T, E, k, 0.1)
        jobs.append({"x": dev(values(rng, (T, cols), 1)), "order": dev(order), "offsets": dev(offsets), "n": m,
                     "host": order, "y": torch.zeros(T * k, cols, device="cuda:0"), "stream": torch.cuda.Stream(),
                     "pos": torch.zeros(T * k, dtype=torch.int32, device="cuda:0"), "out": torch.zeros(T, cols, device="cuda:0"),
                     "codes": torch.zeros(T * k, ref.padded(cols), dtype=torch.int8, device="cuda:0"),
                     "scales": torch.zeros(T * k, device="cuda:0"), "C": torch.zeros(T * k, T * k, device="cuda:0")})
    sync()

    def work(j):
        try:
            for _ in range(20):
                c3.c3_dispatch(j["x"], 1, T, cols, cols, j["order"], j["offsets"], k, E, j["y"], cols, j["pos"], j["stream"])
                c3.c3_combine(j["y"], 1, T, k, cols, cols, j["pos"], None, j["out"], cols, j["stream"])
                c3.c3_i8_dispatch(j["x"], 1, T, cols, cols, j["order"], j["offsets"], k, E, j["codes"], j["scales"],
                                  j["pos"], j["stream"])
                c3.c3_i8_gemm(j["codes"], j["scales"], j["codes"], j["scales"], j["C"], 1, T * k, T * k, cols, T * k,
                              j["stream"])
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    sync()
    assert not bad, bad
    for j in jobs:
        x, order, m = j["x"].cpu().numpy(), j["host"], j["n"]
        np.testing.assert_array_equal(j["y"].cpu().numpy()[:m], ref.sort_rows(x, order, m))
        pos = ref.positions(order, m, T * k).reshape(k, T)
        want, bound = ref.combine(j["y"].cpu().numpy(), pos, None)
        assert (np.abs(j["out"].cpu().numpy() - want) <= bound + ref.HALF[1] * (np.abs(want) + bound)).all()
        A, s = ref.quantize(x)
        A, s = A[order[:m] % T], s[order[:m] % T]
        np.testing.assert_array_equal(j["C"].cpu().numpy()[:m, :m], ref.product(A, s, A, s))


def test_two_streams_and_repeats_give_the_same_bits(c3gpu):
    import torch

    rng = np.random.default_rng(12)
    T, E, k, cols = 500, 16, 4, 1000
    pos, n = plan_of(rng, T, E, k, 0.1)
    y, d, w, p = (dev(a) for a in (values(rng, (T * k, cols), 1), values(rng, (T, cols), 1),
                                   rng.random((T, k)).astype(np.float32), pos))
    sync()
    results = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams * 3:
        out, dy, dw = (torch.zeros(*n_, device="cuda:0") for n_ in ((T, cols), (T * k, cols), (T, k)))
        s.wait_stream(torch.cuda.current_stream())
        c3gpu.c3_combine(y, 1, T, k, cols, cols, p, w, out, cols, s)
        c3gpu.c3_combine_backward(d, 1, T, k, cols, cols, y, cols, p, w, dy, cols, dw, s)
        results.append((out, dy, dw))
    sync()
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))


def test_refusals_that_need_the_device(c3gpu):
    import torch

    c3 = c3gpu
    x, y = torch.zeros(4, 64, device="cuda:0"), torch.zeros(8, 64, device="cuda:0")
    order, pos = torch.zeros(8, dtype=torch.int32, device="cuda:0"), torch.zeros(8, dtype=torch.int32, device="cuda:0")
    offsets = torch.zeros(5, dtype=torch.int32, device="cuda:0")
    with pytest.raises(c3.C3Error, match="device memory"):
        c3.c3_dispatch(torch.zeros(4, 64).data_ptr(), 1, 4, 64, 64, order, offsets, 2, 4, y, 64, pos)
    with pytest.raises(c3.C3Error, match="run past|overlaps"):
        c3.c3_dispatch(x, 1, 4, 64, 1 << 30, order, offsets, 2, 4, y, 64, pos)
    c3.c3_dispatch(x, 1, 0, 64, 64, order, offsets, 2, 4, y, 64, pos)
    c3.c3_combine(y, 1, 0, 2, 64, 64, pos, None, x, 64)
    c3.c3_combine_backward(x, 1, 0, 2, 64, 64, None, 64, pos, None, y, 64, None)
