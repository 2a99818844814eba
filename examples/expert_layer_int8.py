"""A layer of experts with 8-bit integer weights, from the C3 library's entry points alone (torch
holds the memory and applies the activation):

    route -> slot plan -> tokens quantised and sorted by expert -> every expert's up product
          -> activation -> quantise -> every expert's down product -> weighted sum over a token's experts

Between the sort and the sum every buffer is in expert order: what an all-to-all sends and delivers
where the experts are spread over several GPUs. A step has no sizes that the GPU decides, so a decoding
step is captured into a graph once and replayed (`main`).

    python examples/expert_layer_int8.py [tokens]
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from concurrent_gemm_dma_amd import _c3 as c3  # noqa: E402


class Int8:
    """An int8 operand of rows x cols."""

    def __init__(self, rows, cols, device):
        self.rows, self.cols = rows, cols
        codes, _ = c3.c3_i8_bytes(rows, cols)
        self.codes = torch.zeros(codes, dtype=torch.int8, device=device)
        self.scales = torch.zeros(rows, device=device)

    def quantise(self, x):
        """From contiguous bf16 x [rows][cols]."""
        c3.c3_i8_quantize(x, c3.C3_BF16, self.rows, self.cols, self.cols, self.codes, self.scales,
                          torch.cuda.current_stream())
        return self


class ExpertLayer:
    """up [E][F][D] and down [E][D][F] are quantised once, a scale for each output channel; buffers
    are for T tokens."""

    def __init__(self, up, down, T, opts):
        self.E, self.F, self.D = up.shape
        self.T, self.k, self.opts = T, opts.top_k, opts
        E, F, D, S, dev = self.E, self.F, self.D, T * opts.top_k, up.device
        self.S = S
        self.up, self.down = Int8(E * F, D, dev).quantise(up), Int8(E * D, F, dev).quantise(down)
        whole = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
        # rows of no expert are left as they were (zeros, or an earlier step's); no result comes from them
        half = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.idx, self.weights = whole(T, self.k), torch.empty(T, self.k, device=dev)
        self.order, self.offsets, self.pos = whole(S), whole(E + 1), whole(S)
        self.x8, self.h8 = Int8(S, D, dev), Int8(S, F, dev)
        self.h, self.z, self.y = half(S, F), half(S, D), half(T, D)

    def product(self, a, b, out, n):
        c3.c3_i8_gemm_experts(a.codes, a.scales, b.codes, b.scales, self.offsets, out, c3.C3_BF16, self.S, self.E, n,
                              a.cols, n, torch.cuda.current_stream())

    def forward(self, x, logits):
        """bf16 y [T][D] of bf16 x [T][D] and fp32 logits [T][E]; a buffer of the layer's own."""
        T, k, E, D, s = self.T, self.k, self.E, self.D, torch.cuda.current_stream()
        c3.c3_route(logits, c3.C3_F32, T, E, E, self.opts, None, self.idx, self.weights, s)
        c3.c3_route_plan(self.idx, T, k, E, self.order, self.offsets, s)
        c3.c3_i8_dispatch(x, c3.C3_BF16, T, D, D, self.order, self.offsets, k, E, self.x8.codes, self.x8.scales,
                          self.pos, s)
        self.product(self.x8, self.up, self.h, self.F)
        torch.nn.functional.silu(self.h, inplace=True)
        self.h8.quantise(self.h)
        self.product(self.h8, self.down, self.z, D)
        c3.c3_combine(self.z, c3.C3_BF16, T, k, D, D, self.pos, self.weights, self.y, D, s)
        return self.y

    def backward(self, logits, dy):
        """(dz [S][D] in expert order, dlogits [T][E]) of the last forward, from dy [T][D]."""
        T, k, E, D, s = self.T, self.k, self.E, self.D, torch.cuda.current_stream()
        dz, dw, dlogits = torch.zeros_like(self.z), torch.empty_like(self.weights), torch.empty_like(logits)
        c3.c3_combine_backward(dy, c3.C3_BF16, T, k, D, D, self.z, D, self.pos, self.weights, dz, D, dw, s)
        c3.c3_route_backward(logits, c3.C3_F32, T, E, E, self.opts, self.idx, dw, dlogits, E, s)
        return dz, dlogits

    def tokens_gradient(self, dx_rows):
        """The sort's gradient: bf16 dx [T][D] from gradients dx_rows [S][D] of the sorted rows, which a
        training program has from backward's dz by way of the experts' weights."""
        dx = torch.empty_like(self.y)
        c3.c3_combine(dx_rows, c3.C3_BF16, self.T, self.k, self.D, self.D, self.pos, None, dx, self.D,
                      torch.cuda.current_stream())
        return dx


def main(T=8, E=32, D=4096, F=2048, k=4):
    c3.c3_init(0)
    g = torch.Generator(device="cuda:0").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda:0")  # noqa: E731
    layer = ExpertLayer((randn(E, F, D) / D ** 0.5).bfloat16(), (randn(E, D, F) / F ** 0.5).bfloat16(), T,
                        c3.route_opts(c3.C3_SCORE_SOFTMAX, k))
    x, logits = randn(T, D).bfloat16(), randn(T, E)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.forward(x, logits)  # the plan's workspace is allocated outside the capture
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer.forward(x, logits)
    graph.replay()
    torch.cuda.synchronize()
    start, n = time.perf_counter(), 50
    for _ in range(n):
        graph.replay()
    torch.cuda.synchronize()
    print(f"{T} tokens, {E} experts of {D} x {F}, {k} each: {(time.perf_counter() - start) / n * 1e6:.1f} us a step")
    dz, dlogits = layer.backward(logits, randn(T, D).bfloat16())
    # the experts' weights are quantised and have no gradient here: dz stands in for the sorted rows' own
    print("gradients: rows", tuple(dz.shape), "router", tuple(dlogits.shape),
          "and, as shapes go, rows brought back to tokens", tuple(layer.tokens_gradient(dz).shape))
    torch.cuda.synchronize()


if __name__ == "__main__":
    main(*map(int, sys.argv[1:2]))
