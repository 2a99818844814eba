"""examples/expert_layer_int8.py over several steps: a layer keeps its buffers, so rows that no expert has
in a step hold those of an earlier one. Nothing that a step gives comes from them."""
import numpy as np
import pytest

from test_gpu_expert_layer_int8 import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,D,F,k", [(37, 6, 520, 264, 3), (6000, 8, 640, 256, 4)])
def test_steps_with_fewer_and_more_tokens_routed(c3gpu, T, E, D, F, k):
    import torch

    m, c3 = example(), c3gpu
    g = torch.Generator(device="cuda:0").manual_seed(T)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda:0")  # noqa: E731
    up, down = (randn(E, F, D) / D ** 0.5).bfloat16(), (randn(E, D, F) / F ** 0.5).bfloat16()
    new = lambda: m.ExpertLayer(up, down, T, c3.route_opts(c3.C3_SCORE_SOFTMAX, k))  # noqa: E731
    kept = new()
    for masked in (0.0, 0.6, 0.1, 1.0, 0.3):
        x, logits, dy = randn(T, D).bfloat16(), randn(T, E), randn(T, D).bfloat16()
        logits[torch.rand(T, generator=g, device="cuda:0") < masked] = -np.inf
        fresh = new()
        results = []
        for layer in (kept, fresh):
            y = layer.forward(x, logits).clone()
            dz, dlogits = layer.backward(logits, dy)
            results.append([y, dz, dlogits, layer.tokens_gradient(dz), layer.pos, layer.offsets, layer.weights])
        torch.cuda.synchronize()
        n = int(fresh.offsets[-1])
        assert n == k * int((logits[:, 0] > -np.inf).sum())
        for a, b in zip(*results):
            assert torch.equal(a, b)
        assert torch.equal(kept.z[:n], fresh.z[:n])


def test_what_main_says_of_its_gradients(c3gpu, capsys):
    example().main(3, 8, 512, 256, 2)
    out = capsys.readouterr().out
    assert "rows brought back to tokens (3, 512)" in out
