"""Routing on the GPU against the 64-bit definitions of layer_ref: choices and plans exactly,
weights and gradients within derived bounds, on masks, ties, infinities and NaN; the three calls
in a captured graph; refusals that need the device."""
import numpy as np
import pytest

import layer_ref as ref

pytestmark = pytest.mark.gpu
KINDS = {"softmax": 0, "sigmoid": 1}


def dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")


def held(x, dtype, ld):
    """x with row stride ld in the type, NaN past the experts."""
    import torch

    h = np.full((x.shape[0], ld), np.nan, np.float32)
    h[:, :x.shape[1]] = x
    return dev(h).to(torch.bfloat16 if dtype == 0 else torch.float32)


def run(c3, x, dtype, k, kind="softmax", groups=1, top_groups=1, group_top=1, bias=None, renorm=True, scale=1.0,
        ld=None):
    import torch

    T, E = x.shape
    idx = torch.full((T + 1, k), -9, dtype=torch.int32, device="cuda:0")
    w = torch.full((T + 1, k), -9.0, device="cuda:0")
    o = c3.route_opts(KINDS[kind], k, groups, top_groups, group_top, renorm, scale)
    c3.c3_route(held(x, dtype, ld or E), dtype, T, E, ld or E, o, None if bias is None else dev(bias), idx, w)
    torch.cuda.synchronize()
    assert (idx[T] == -9).all().item() and (w[T] == -9).all().item()
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy()


def logits(rng, T, E, dtype, masked=0.0):
    x = (1.5 * rng.normal(0, 1, (T, E)) + 0.5 * rng.normal(0, 1, E)).astype(np.float32)
    if dtype == 0:
        x = ref.bf16_round(x)
    if masked:
        x[rng.random((T, E)) < masked] = -np.inf
        x[rng.random(T) < 0.1] = -np.inf
    return x


def weights_close(x, idx, got, want, scale=1.0):
    """Half a step of the rounding to fp32, and of each of the few fp32 steps before it: a rounded
    exponent of size r shifts e^r by r half steps, and sums of non-negative terms add one each."""
    with np.errstate(invalid="ignore"):
        l = np.array([ref.clean(r) for r in x])
        span = np.zeros((len(x), 1))
        for t in range(len(x)):
            fin = l[t][l[t] > -np.inf]
            span[t] = min(fin.max() - fin.min(), 200.0) if len(fin) else 0.0
    limit = (span + idx.shape[1] + 24) * 2.0 ** -24 * np.abs(want) + 2.0 ** -126
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


CASES = [dict(T=1, E=256, k=8, kind="sigmoid", groups=8, top_groups=4, group_top=2, bias=True),
         dict(T=1, E=1, k=1), dict(T=3, E=4, k=4, kind="sigmoid"), dict(T=130, E=128, k=8),
         dict(T=257, E=64, k=6, renorm=False), dict(T=65, E=65, k=3, bias=True, renorm=False),
         dict(T=100, E=160, k=6, groups=8, top_groups=3), dict(T=100, E=160, k=6, groups=8, top_groups=3, group_top=2),
         dict(T=100, E=252, k=8, groups=4, top_groups=1, group_top=2, bias=True, kind="softmax"),
         dict(T=50, E=256, k=8, kind="sigmoid", renorm=False, scale=2.5), dict(T=33, E=384, k=10, bias=True),
         dict(T=20, E=1024, k=64, kind="sigmoid", bias=True), dict(T=20, E=1000, k=16, groups=8, top_groups=4),
         dict(T=64, E=64, k=5, groups=64, top_groups=9, group_top=2, kind="sigmoid")]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_route(c3gpu, case, dtype, masked):
    c = dict(case)
    T, E, k = c.pop("T"), c.pop("E"), c.pop("k")
    rng = np.random.default_rng(T + 3 * E + k)
    x = logits(rng, T, E, dtype, masked)
    c["bias"] = (0.1 * rng.normal(0, 1, E)).astype(np.float32) if c.get("bias") else None
    idx, w = run(c3gpu, x, dtype, k, ld=E + T % 3, **c)
    want_i, want_w = ref.route(x, k, **c)
    np.testing.assert_array_equal(idx, want_i)
    weights_close(x, idx, w, want_w)


# batches of over 2048 tokens take another arrangement of the lanes
LARGE = [dict(T=2049, E=17, k=3, kind="sigmoid"), dict(T=2051, E=128, k=8), dict(T=2050, E=100, k=16, renorm=False),
         dict(T=2049, E=256, k=8, kind="sigmoid", groups=8, top_groups=4, group_top=2, bias=True),
         dict(T=2300, E=252, k=7, groups=7, top_groups=3, group_top=2, kind="sigmoid"),
         dict(T=4098, E=256, k=8, kind="sigmoid", groups=8, top_groups=4, group_top=2, bias=True),
         dict(T=4097, E=250, k=9, bias=True), dict(T=4099, E=205, k=5, groups=5, top_groups=2),
         dict(T=2050, E=48, k=2, groups=16, top_groups=5, bias=True),
         dict(T=2049, E=30, k=4, groups=3, top_groups=2, group_top=2),
         dict(T=2049, E=256, k=20, groups=2, top_groups=1, bias=True), dict(T=2049, E=320, k=4),
         dict(T=2049, E=66, k=2, groups=33, top_groups=7, group_top=2, kind="sigmoid", bias=True)]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("case", LARGE, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_route_large_batches(c3gpu, case, dtype):
    test_route(c3gpu, case, dtype, 0.1)


@pytest.mark.parametrize("bias", [False, True])
def test_route_large_batch_ties_and_special_values(c3gpu, bias):
    rng = np.random.default_rng(4)
    T, E, k = 2100, 96, 8
    x = np.round(rng.normal(0, 1, (T, E)) * 2).astype(np.float32) / 2
    x[::3] = rng.choice(np.array([np.inf, -np.inf, np.nan, np.finfo(np.float32).min, 0.0, -0.0, 1e-45, -1e-45, 200.0],
                                 np.float32), (T // 3, E))
    b = (rng.integers(-2, 3, E) / 8).astype(np.float32) if bias else None
    for kind in ("softmax", "sigmoid"):
        # sums of two scores with a bias can tie up to their last bits: not compared here
        for groups, top, gt in ((1, 1, 1), (8, 3, 1 if bias else 2)):
            idx, w = run(c3gpu, x, 1, k, kind, groups, top, gt, b)
            want_i, want_w = ref.route(x, k, kind, groups, top, gt, b)
            np.testing.assert_array_equal(idx, want_i)
            weights_close(x, idx, w, want_w)


@pytest.mark.parametrize("E,groups", [(1020, 17), (990, 33), (1023, 3), (1024, 64)])
def test_route_many_experts_in_groups(c3gpu, E, groups):
    rng = np.random.default_rng(E)
    x = logits(rng, 40, E, 1, 0.1)
    b = (0.1 * rng.normal(0, 1, E)).astype(np.float32)
    for bias in (None, b):
        idx, w = run(c3gpu, x, 1, 12, "sigmoid", groups, 2, 2, bias)
        want_i, want_w = ref.route(x, 12, "sigmoid", groups, 2, 2, bias)
        np.testing.assert_array_equal(idx, want_i)
        weights_close(x, idx, w, want_w)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_ties_and_near_ties(c3gpu, kind, bias):
    """Equal values go to the lower index, and scores a rounding of fp32 apart are told apart."""
    rng = np.random.default_rng(2)
    T, E, k = 200, 96, 8
    x = np.round(rng.normal(0, 1, (T, E)) * 2).astype(np.float32) / 2  # many equal logits
    x[::2] += (rng.integers(-3, 4, (T // 2, E)) * 2.0 ** -23).astype(np.float32)  # a few steps apart
    b = (rng.integers(-2, 3, E) / 8).astype(np.float32) if bias else None
    for groups, top, gt in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        idx, _ = run(c3gpu, x, 1, k, kind, groups, top, gt, b)
        want = ref.route(x, k, kind, groups, top, gt, b)[0]
        np.testing.assert_array_equal(idx, want)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_special_values(c3gpu, kind, renorm):
    """Tokens without experts, one expert, infinities, NaN, the type's lowest value, scores that
    underflow and that saturate; a bias of -infinity takes an expert out."""
    low = float(np.finfo(np.float32).min)
    x = np.zeros((10, 70), np.float32)
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = -np.inf
    x[2, 69] = -3
    x[3, 7], x[3, 8] = np.inf, np.inf
    x[4, 5] = np.nan
    x[5] = low
    x[6] = np.linspace(-300, -200, 70)
    x[7] = np.linspace(200, 300, 70)
    x[8] = np.linspace(-80, 80, 70)
    x[9] = low
    x[9, 3], x[9, 60] = 1.0, 2.0
    idx, w = run(c3gpu, x, 1, 4, kind, renorm=renorm)
    want_i, want_w = ref.route(x, 4, kind, renorm=renorm)
    np.testing.assert_array_equal(idx, want_i)
    weights_close(x, idx, w, want_w)
    assert (idx[:2] == -1).all() and (w[:2] == 0).all() and list(idx[2]) == [69, -1, -1, -1]
    bias = np.zeros(70, np.float32)
    bias[:60] = -np.inf
    idx, w = run(c3gpu, x, 1, 4, kind, bias=bias, renorm=renorm)
    want_i, want_w = ref.route(x, 4, kind, bias=bias, renorm=renorm)
    np.testing.assert_array_equal(idx, want_i)
    weights_close(x, idx, w, want_w)


def gradient(c3, x, dtype, idx, dw, kind, renorm, scale, ld=None):
    import torch

    T, E = x.shape
    out = torch.full((T + 1, ld or E), -9.0, dtype=torch.bfloat16 if dtype == 0 else torch.float32, device="cuda:0")
    o = c3.route_opts(KINDS[kind], idx.shape[1], renormalize=renorm, scale=scale)
    c3.c3_route_backward(held(x, dtype, ld or E), dtype, T, E, ld or E, o, dev(idx), dev(dw), out, ld or E)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    assert (got[T] == -9).all() and (got[:, E:] == -9).all()
    return got[:T, :E]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 8), (130, 64, 6), (67, 200, 3), (33, 256, 8), (9, 1000, 40)])
def test_route_backward(c3gpu, T, E, k, kind, renorm, dtype):
    rng = np.random.default_rng(T + E)
    x = logits(rng, T, E, dtype, 0.2 if T > 5 else 0.0)
    idx, _ = ref.route(x, k, kind)
    if T > 30:
        idx[3], idx[4, 1], idx[5, 0] = -1, E, -7   # absent entries of every sort
        idx[6, 1] = idx[6, 0]                      # an expert named twice
        idx[7, 0] = int(np.argmin(np.where(np.isneginf(x[7]), -1e30, x[7])))  # maybe out of reach
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    got = gradient(c3gpu, x, dtype, idx, dw, kind, renorm, 1.5, ld=E + 3)
    want, size = ref.route_gradient(x, idx, dw, kind, renorm, 1.5)
    half = 2.0 ** -8 if dtype == 0 else 2.0 ** -24
    # exponents of size below 40 and sums of up to E terms, each rounded in fp32
    limit = (40 + 24 + k + E / 8) * 2.0 ** -24 * size + half * np.abs(want) + 2.0 ** -126
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k,dtype", [(4100, 17, 3, 0), (4101, 100, 8, 1), (4099, 201, 16, 0)])
def test_route_backward_large_batches(c3gpu, T, E, k, kind, renorm, dtype):
    test_route_backward(c3gpu, T, E, k, kind, renorm, dtype)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(c3gpu, kind, renorm):
    """dlogits . v is the slope of the forward's weights along v."""
    rng = np.random.default_rng(11)
    T, E, k, h = 40, 32, 4, 2.0 ** -7
    x = rng.normal(0, 1, (T, E)).astype(np.float32)
    x[np.arange(T)[:, None], np.argsort(rng.random((T, E)), 1)[:, :k]] += 3  # the choice holds along v
    v = rng.choice([-1.0, 1.0], (T, E)).astype(np.float32)
    idx, _ = run(c3gpu, x, 1, k, kind, renorm=renorm)
    up_i, up = run(c3gpu, x + np.float32(h) * v, 1, k, kind, renorm=renorm)
    dn_i, dn = run(c3gpu, x - np.float32(h) * v, 1, k, kind, renorm=renorm)
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    d = gradient(c3gpu, x, 1, idx, dw, kind, renorm, 1.0)
    same = (np.sort(up_i, 1) == np.sort(idx, 1)).all(1) & (np.sort(dn_i, 1) == np.sort(idx, 1)).all(1)
    assert same.sum() > T // 2
    for t in np.flatnonzero(same):
        f = [sum(dw[t, j] * w[t, list(i[t]).index(idx[t, j])] for j in range(k)) for i, w in ((up_i, up), (dn_i, dn))]
        # truncation h^2 / 6 times a third derivative of at most 8 per weight, rounding 32 half
        # steps of the weights over 2 h
        limit = np.abs(dw[t]).sum() * (h * h * 8 / 6 + 64 * 2.0 ** -24 / (2 * h))
        assert abs((f[0] - f[1]) / (2 * h) - (d[t] * v[t]).sum()) <= limit


@pytest.mark.parametrize("T,E,k", [(0, 5, 2), (1, 256, 8), (7, 3, 2), (511, 8, 8), (513, 1024, 8), (700, 24, 6),
                                   (5000, 1, 1), (9001, 256, 8), (30000, 128, 4), (70001, 1000, 3)])
def test_plan(c3gpu, T, E, k):
    import torch

    rng = np.random.default_rng(T)
    idx = np.minimum((E * rng.random((T, k)) ** 3).astype(np.int32), E - 1)  # uneven
    idx[rng.random((T, k)) < 0.1] = -1
    if T > 2:
        idx[0, 0], idx[2, 0] = E, 1 << 30
    order = torch.full((T * k + 1,), -9, dtype=torch.int32, device="cuda:0")
    offsets = torch.full((E + 2,), -9, dtype=torch.int32, device="cuda:0")
    c3gpu.c3_route_plan(dev(idx), T, k, E, order, offsets)
    torch.cuda.synchronize()
    want = ref.plan(idx, E)
    np.testing.assert_array_equal(order.cpu().numpy(), np.append(want[0], -9))
    np.testing.assert_array_equal(offsets.cpu().numpy(), np.append(want[1], -9))


def test_route_in_a_captured_graph(c3gpu):
    """Routing, plan, quantisation, experts' products and the gradient recorded once and replayed
    on new inputs, with eager work between; each replay equals the eager calls bit for bit."""
    import torch

    c3, T, E, k, N, K = c3gpu, 1100, 16, 4, 200, 320
    g = torch.Generator(device="cuda:0").manual_seed(1)
    make = lambda *s: torch.randn(*s, generator=g, device="cuda:0")  # noqa: E731
    x, logit, dw = make(T, K), make(T, E), make(T, k)
    o = c3.route_opts(c3.C3_SCORE_SIGMOID, k)
    empty = lambda n, t=torch.uint8: torch.zeros(n, dtype=t, device="cuda:0")  # noqa: E731
    b, sb = empty(c3.c3_mx4_bytes(E * N, K)[0]), empty(c3.c3_mx4_bytes(E * N, K)[1])
    c3.c3_mx4_quantize(make(E * N, K), 1, E * N, K, K, False, 0, b, sb)

    def buffers():
        nc, ns = c3.c3_mx4_bytes(T, K)
        return dict(a=empty(nc), sa=empty(ns), idx=empty(T * k, torch.int32), w=empty(T * k, torch.float32),
                    order=empty(T * k, torch.int32), offsets=empty(E + 1, torch.int32),
                    C=empty(T * k * N, torch.float32), d=empty(T * E, torch.float32))

    def step(m, s):
        c3.c3_route(logit, 1, T, E, E, o, None, m["idx"], m["w"], s)
        c3.c3_route_plan(m["idx"], T, k, E, m["order"], m["offsets"], s)
        c3.c3_mx4_quantize(x, 1, T, K, K, False, 0, m["a"], m["sa"], s)
        c3.c3_mx4_gemm_experts(m["a"], m["sa"], T, b, sb, m["order"], m["offsets"], m["w"], m["C"], 1, T, k, E, N, K,
                               N, s)
        c3.c3_route_backward(logit, 1, T, E, E, o, m["idx"], dw, m["d"], E, s)

    held, eager = buffers(), buffers()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(c3.C3Error) as e:  # the plan's workspace cannot be allocated while capturing
        with torch.cuda.graph(graph, stream=stream):
            c3.c3_route_plan(held["idx"], T, k, E, held["order"], held["offsets"], stream)
    assert e.value.status == c3.C3_E_UNSUPPORTED
    torch.cuda.synchronize()
    step(held, stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(held, stream)
    for i in range(3):
        logit.copy_(make(T, E))
        x.copy_(make(T, K))
        dw.copy_(make(T, k))
        for t in held.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(eager, None)
        torch.cuda.synchronize()
        for n in held:
            assert torch.equal(held[n], eager[n]), (i, n)


@pytest.mark.parametrize("T,E,k", [(64, 1024, 1), (65, 9, 1), (8, 5, 8), (4096, 300, 1), (4097, 300, 1),
                                   (262145, 64, 1), (40000, 1024, 8)])
def test_plan_at_the_borders_of_its_kernels(c3gpu, T, E, k):
    test_plan(c3gpu, T, E, k)


def large_plan(seed, T=20000, E=100, k=3):
    """(idx, buffers, want) of a plan above 4096 slots, on the device."""
    import torch

    idx = np.random.default_rng(seed).integers(-1, E, (T, k)).astype(np.int32)
    whole = lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda:0")  # noqa: E731
    return dev(idx), (whole(T * k), whole(E + 1)), ref.plan(idx, E), (T, k, E)


def planned(buffers, want):
    return all((b.cpu().numpy() == w).all() for b, w in zip(buffers, want))


def test_plan_on_the_per_thread_stream(c3gpu):
    """One handle, a stream of its own in each host thread: the plans may overlap."""
    import threading

    import torch

    per_thread = 2  # hipStreamPerThread
    work = [[large_plan(10 * t + i) for i in range(6)] for t in range(4)]
    torch.cuda.synchronize()
    failed = []

    def plan(mine):
        try:
            for _ in range(5):
                for idx, buffers, _, size in mine:
                    c3gpu.c3_route_plan(idx, *size, *buffers, per_thread)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=plan, args=(mine,)) for mine in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    assert all(planned(buffers, want) for mine in work for _, buffers, want, _ in mine)


def test_plan_beside_the_replay_of_a_graph(c3gpu):
    """Eager plans on the stream a graph was captured on, while it is replayed on another."""
    import torch

    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    idx, buffers, want, size = large_plan(1)
    e_idx, e_buffers, e_want, _ = large_plan(2)
    torch.cuda.synchronize()
    c3gpu.c3_route_plan(idx, *size, *buffers, stream)  # the workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(20):
            c3gpu.c3_route_plan(idx, *size, *buffers, stream)
    for _ in range(4):
        for b in buffers + e_buffers:
            b.fill_(-9)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            graph.replay()
        for _ in range(20):
            c3gpu.c3_route_plan(e_idx, *size, *e_buffers, stream)
        torch.cuda.synchronize()
        assert planned(buffers, want) and planned(e_buffers, e_want)


def test_destroyed_streams_give_their_plan_workspace_back(c3gpu):
    import torch

    idx, buffers, want, size = large_plan(3)
    torch.cuda.synchronize()

    def taken(n, plan):
        """Device memory that n streams leave behind."""
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        for _ in range(n):
            s = c3gpu.c3_stream_create()
            if plan:
                c3gpu.c3_route_plan(idx, *size, *buffers, s)
            c3gpu.c3_stream_destroy(s)
        torch.cuda.synchronize()
        return free - torch.cuda.mem_get_info()[0]

    taken(1, True)
    streams = taken(20, False)
    assert taken(20, True) - streams < 10 * c3gpu.C3_PLAN_WORKSPACE_BYTES
    assert planned(buffers, want)


def test_route_of_more_tokens_than_a_launch_takes(c3gpu):
    """2^26 tokens and some: each repeats one of 999 tokens, and gets that token's choice and gradient."""
    import torch

    rng = np.random.default_rng(6)
    T, E, k, n = (1 << 26) + 77, 4, 2, 999
    x = logits(rng, n, E, 0, 0.1)
    dw = rng.normal(0, 1, (n, k)).astype(np.float32)
    idx, w = run(c3gpu, x, 0, k)
    few = gradient(c3gpu, x, 0, idx, dw, "softmax", True, 1.0)
    want_i, want_w = ref.route(x, k)
    np.testing.assert_array_equal(idx, want_i)
    weights_close(x, idx, w, want_w)

    again = lambda v: dev(v).repeat(T // n + 1, 1)[:T]  # noqa: E731
    all_x, all_dw = again(x).bfloat16(), again(dw)
    all_idx = torch.full((T + 1, k), -9, dtype=torch.int32, device="cuda:0")
    all_w = torch.full((T + 1, k), -9.0, device="cuda:0")
    d = torch.full((T + 1, E), -9.0, dtype=torch.bfloat16, device="cuda:0")
    o = c3gpu.route_opts(top_k=k)
    c3gpu.c3_route(all_x, 0, T, E, E, o, None, all_idx, all_w)
    c3gpu.c3_route_backward(all_x, 0, T, E, E, o, all_idx, all_dw, d, E)
    torch.cuda.synchronize()
    assert (all_idx[T] == -9).all().item() and (all_w[T] == -9).all().item() and (d[T] == -9).all().item()
    assert torch.equal(all_idx[:T], again(idx))
    # another arrangement of the lanes adds in another order: both within the bound of the few
    assert ((all_w[:T] - again(w)).abs() <= (40 + k) * 2.0 ** -23).all().item()
    limit = again((2.0 ** -7 * np.abs(few) + 140 * 2.0 ** -23 * np.abs(dw).sum(1, keepdims=True)).astype(np.float32))
    assert ((d[:T].float() - again(few.astype(np.float32))).abs() <= limit).all().item()
    del all_x, all_dw, all_idx, all_w, d, limit
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_where_the_bias_cancels_the_score(c3gpu, kind):
    """Biases that are the scores' negatives rounded to fp32: what is left is a rounding of the
    score, and a choice may only be out of order by the stated 2^-42 of |s + bias| and s."""
    rng = np.random.default_rng(13)
    T, E, k = 300, 64, 12
    base = rng.normal(0, 1.5, E).astype(np.float32)
    x = np.tile(base, (T, 1))
    if kind == "sigmoid":
        x = (x * (1 + rng.integers(-2, 3, (T, E)) * 2.0 ** -23)).astype(np.float32)
    else:
        x[1::2, 3] += (rng.integers(-2, 3, T // 2) * 2.0 ** -23).astype(np.float32)
    wide = x.astype(np.longdouble)
    if kind == "sigmoid":
        s = 1 / (1 + np.exp(-wide))
    else:
        s = np.exp(wide - wide.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    bias = (-s[0]).astype(np.float32)
    idx, _ = run(c3gpu, x, 1, k, kind, bias=bias)
    v = s + bias.astype(np.longdouble)
    slack = 2.0 ** -42 * (np.abs(v) + s)
    for t in range(T):
        chosen = idx[t]
        assert len(set(chosen)) == k and (chosen >= 0).all()
        rest = np.setdiff1d(np.arange(E), chosen)
        for a, b in [*zip(chosen[:-1], chosen[1:]), *((chosen[-1], e) for e in rest)]:
            assert v[t, a] >= v[t, b] - max(slack[t, a], slack[t, b]), (t, a, b)


def repeated(x, T):
    return np.resize(x, (T, x.shape[1]))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("case", [
    dict(T=24580, E=256, k=8, kind="sigmoid", groups=8, top_groups=4, group_top=2, bias=True),
    dict(T=24579, E=252, k=5, groups=4, top_groups=2, bias=True), dict(T=7171, E=250, k=9, bias=True),
    dict(T=7170, E=201, k=16, kind="sigmoid", bias=True, renorm=False), dict(T=4097, E=255, k=7),
    dict(T=2305, E=256, k=8, kind="sigmoid", groups=8, top_groups=4, group_top=2), dict(T=2306, E=160, k=6, groups=8,
                                                                                       top_groups=3)],
    ids=lambda c: "-".join(str(v) for v in c.values()))
def test_route_four_tokens_a_wave(c3gpu, case, dtype):
    """Past the batch from which 129 to 256 experts take four tokens a wave, of each form."""
    c = dict(case)
    T, E, k = c.pop("T"), c.pop("E"), c.pop("k")
    rng = np.random.default_rng(T + E)
    few = logits(rng, 301, E, dtype, 0.1)
    c["bias"] = (0.1 * rng.normal(0, 1, E)).astype(np.float32) if c.get("bias") else None
    idx, w = run(c3gpu, repeated(few, T), dtype, k, ld=E + 1, **c)
    want_i, want_w = ref.route(few, k, **c)
    np.testing.assert_array_equal(idx, repeated(want_i, T))
    weights_close(few, want_i, w[:301], want_w)
    weights_close(repeated(few, T)[-301:], want_i, w[-301:], repeated(want_w, T)[-301:])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,E,k,kind,renorm", [
    (3075, 33, 6, "sigmoid", False), (4099, 64, 16, "softmax", False), (5122, 127, 8, "softmax", True),
    (6658, 100, 8, "softmax", False), (6147, 256, 8, "sigmoid", True), (10243, 255, 16, "softmax", False)])
def test_route_backward_four_tokens_a_wave(c3gpu, T, E, k, kind, renorm, dtype):
    rng = np.random.default_rng(T + E)
    few = logits(rng, 301, E, dtype, 0.1)
    idx, _ = ref.route(few, k, kind)
    idx[3], idx[4, 1], idx[5, 0] = -1, E, -7
    idx[6, 1] = idx[6, 0]
    dw = rng.normal(0, 1, (301, k)).astype(np.float32)
    got = gradient(c3gpu, repeated(few, T), dtype, repeated(idx, T), repeated(dw, T), kind, renorm, 1.5, ld=E + 3)
    want, size = (repeated(v, T) for v in ref.route_gradient(few, idx, dw, kind, renorm, 1.5))
    half = 2.0 ** -8 if dtype == 0 else 2.0 ** -24
    # as in test_route_backward
    limit = (40 + 24 + k + E / 8) * 2.0 ** -24 * size + half * np.abs(want) + 2.0 ** -126
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
