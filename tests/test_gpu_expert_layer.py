"""examples/expert_layer.py: the layer's output and gradients against the same layer in 64 bits on
the values that its 4-bit operands stand for."""
import importlib.util
import os

import numpy as np
import pytest

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8  # half a step, relative


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def decoded(pair, rows, cols):
    codes, scales = (t.cpu().numpy().reshape(rows, -1) for t in pair)
    return ref.values(codes, scales, cols)


@pytest.mark.parametrize("T,E,D,F,k", [(1, 8, 256, 320, 2), (37, 6, 520, 264, 3), (700, 5, 384, 512, 2)])
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
    y = layer.forward(x, logits).double().cpu().numpy()
    dlogits = layer.router_gradient(logits, dy).double().cpu().numpy()
    torch.cuda.synchronize()

    idx, w = ref.route(logits.cpu().numpy(), k)
    np.testing.assert_array_equal(layer.idx.cpu().numpy(), idx)
    A, H = decoded(layer.x4, T, D), decoded(layer.h4, T * k, F)
    U, V = decoded(layer.up, E * F, D).reshape(E, F, D), decoded(layer.down, E * D, F).reshape(E, D, F)
    h, h_bound = np.zeros((T * k, F)), np.zeros((T * k, F))
    z, z_bound = np.zeros((T * k, D)), np.zeros((T * k, D))
    for t in range(T):
        for j in range(k):
            if idx[t, j] >= 0:
                s = j * T + t
                p, b = ref.product(A[t:t + 1], U[idx[t, j]])
                h[s], h_bound[s] = p[0], b[0]
                p, b = ref.product(H[s:s + 1], V[idx[t, j]])
                z[s], z_bound[s] = p[0], b[0]
    # the activation: its slope is at most 1.1; two roundings to bf16 and an exponential in fp32
    silu = h / (1 + np.exp(-h))
    got_h = layer.h.double().cpu().numpy()
    limit = 1.1 * (h_bound + BF16 * (np.abs(h) + h_bound)) + 1.1 * BF16 * np.abs(silu) + 16 * 2.0 ** -24 * np.abs(h)
    limit += 2.0 ** -126
    assert (np.abs(got_h - silu) <= limit).all()
    # the sum over a token's experts: each rounded to bf16, added in fp32, rounded to bf16
    wz = w.T[..., None] * z.reshape(k, T, D)
    each = np.abs(wz) * (BF16 + 40 * 2.0 ** -24) + w.T[..., None] * z_bound.reshape(k, T, D) * 1.01
    want, bound = wz.sum(0), each.sum(0) + k * 2.0 ** -24 * np.abs(wz).sum(0)
    limit = bound + BF16 * (np.abs(want) + bound) + 2.0 ** -126
    assert (np.abs(y - want) <= limit).all()
    # dw of each choice (bf16 outputs times dy, added in fp32), then the routing's gradient
    d = dy.double().cpu().numpy()
    dw = (z.reshape(k, T, D) * d).sum(-1).T
    dw_bound = ((np.abs(z) * BF16 + z_bound * 1.01).reshape(k, T, D) * np.abs(d)).sum(-1).T
    dw_bound += (D + 4) * 2.0 ** -24 * (np.abs(z).reshape(k, T, D) * np.abs(d)).sum(-1).T
    want, size = ref.route_gradient(logits.cpu().numpy(), idx, dw)
    moved = ref.route_gradient(logits.cpu().numpy(), idx, dw_bound)[1]  # the terms' size bounds their change
    limit = moved + (64 + k + E / 8) * 2.0 ** -24 * (size + moved) + 2.0 ** -126
    assert (np.abs(dlogits - want) <= limit).all()


@pytest.mark.parametrize("T,n,m_", [(1, 5, 3), (100, 130, 70), (1000, 300, 520)])
def test_weight_gradient(c3gpu, T, n, m_):
    import torch

    m = example()
    g = torch.Generator(device="cuda:0").manual_seed(T)
    dy, x = (torch.randn(T, c, generator=g, device="cuda:0").bfloat16() for c in (n, m_))
    got = m.weight_gradient(dy, x).double().cpu().numpy()
    a, b = (ref.values(*ref.quantize(np.ascontiguousarray(t.float().cpu().numpy().T), True), T) for t in (dy, x))
    want, bound = ref.product(a, b)
    assert (np.abs(got - want) <= bound + 2.0 ** -126).all()


def test_decoding_step_in_a_graph(c3gpu, capsys):
    example().main(3, 8, 512, 256, 2)
    assert "us a step" in capsys.readouterr().out
