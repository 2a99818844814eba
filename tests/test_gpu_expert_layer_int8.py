"""examples/expert_layer_int8.py: the operators in a run, each against its definition on what the
device handed it, and the layer's output and gradients against the same layer in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest

import layer_ref
import sort_ref as ref

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8  # half a step, relative


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer_int8.py")
    spec = importlib.util.spec_from_file_location("expert_layer_int8", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def codes_of(a):
    return a.codes.cpu().numpy().reshape(a.rows, -1), a.scales.cpu().numpy()


def floats(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("T,E,D,F,k", [(1, 8, 256, 320, 2), (37, 6, 520, 264, 3), (700, 5, 384, 512, 2), (2000, 20, 640, 130, 4)])
def test_layer(c3gpu, T, E, D, F, k):
    import torch

    m, c3 = example(), c3gpu
    g = torch.Generator(device="cuda:0").manual_seed(T)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda:0")  # noqa: E731
    layer = m.ExpertLayer((randn(E, F, D) / D ** 0.5).bfloat16(), (randn(E, D, F) / F ** 0.5).bfloat16(), T,
                          c3.route_opts(c3.C3_SCORE_SOFTMAX, k))
    x, logits, dy = randn(T, D).bfloat16(), randn(T, E), randn(T, D).bfloat16()
    if T > 30:
        logits[5] = -np.inf  # a token without experts
        logits[6, 1:] = -np.inf  # and one with a single expert
    torch.cuda.synchronize()
    y = floats(layer.forward(x, logits))
    dz, dlogits = layer.backward(logits, dy)
    dx = floats(layer.tokens_gradient(dz))
    torch.cuda.synchronize()
    dz, dlogits = floats(dz), dlogits.double().cpu().numpy()

    idx, w = layer_ref.route(logits.cpu().numpy(), k)
    np.testing.assert_array_equal(layer.idx.cpu().numpy(), idx)
    order, offsets = ref.plan(idx, E)
    n, S = int(offsets[-1]), T * k
    pos = ref.positions(order, n, S).reshape(k, T)
    np.testing.assert_array_equal(layer.pos.cpu().numpy(), pos.reshape(-1))
    # tokens quantised and sorted; both products bit for bit, of the codes that went into them
    A, sA = codes_of(layer.x8)
    want = ref.quantize(floats(x))
    np.testing.assert_array_equal(A[:n], want[0][order[:n] % T])
    np.testing.assert_array_equal(sA[:n], want[1][order[:n] % T])
    H, sH = codes_of(layer.h8)
    want = ref.quantize(floats(layer.h))
    np.testing.assert_array_equal(H, want[0])
    np.testing.assert_array_equal(sH, want[1])
    (U, sU), (V, sV) = codes_of(layer.up), codes_of(layer.down)
    got_h, z = floats(layer.h), floats(layer.z)
    for e in range(E):
        p = slice(offsets[e], offsets[e + 1])
        h = ref.rounded(ref.product(A[p], sA[p], U[e * F:e * F + F], sU[e * F:e * F + F]), 0).astype(np.float64)
        silu = h / (1 + np.exp(-h))
        # torch's: an exponential and a quotient in fp32, one rounding to bf16
        assert (np.abs(got_h[p] - silu) <= BF16 * np.abs(silu) + 16 * 2.0 ** -24 * np.abs(h) + 2.0 ** -126).all()
        np.testing.assert_array_equal(z[p], ref.rounded(ref.product(H[p], sH[p], V[e * D:e * D + D], sV[e * D:e * D + D]), 0))
    assert not z[n:].any() and not got_h[n:].any()
    # the sum: weights as the device has them are within 2^-20 of the definition's
    wd = layer.weights.cpu().numpy()
    assert (np.abs(wd - w) <= 2.0 ** -20 * w).all()
    out, bound = ref.combine(z, pos, wd)
    assert (np.abs(y - out) <= bound + BF16 * (np.abs(out) + bound)).all()
    # gradients of the rows, the weights, the logits and, back through the sort, of the tokens
    d, written, dw, bound = ref.combine_gradient(floats(dy), z, pos, wd)
    assert (np.abs(dz - d) <= (BF16 + 2.0 ** -24) * 1.01 * np.abs(d) + ref.TINY).all() and not dz[~written].any()
    want, size = layer_ref.route_gradient(logits.cpu().numpy(), idx, dw)
    moved = layer_ref.route_gradient(logits.cpu().numpy(), idx, bound)[1]  # the terms' size bounds their change
    limit = moved + (64 + k + E / 8) * 2.0 ** -24 * (size + moved) + 2.0 ** -126
    assert (np.abs(dlogits - want) <= limit).all()
    want, bound = ref.combine(dz, pos, None)
    assert (np.abs(dx - want) <= bound + BF16 * (np.abs(want) + bound)).all()


def test_decoding_step_in_a_graph(c3gpu, capsys):
    example().main(3, 8, 512, 256, 2)
    out = capsys.readouterr().out
    assert "us a step" in out and "tokens (3, 512)" in out
