"""A layer of experts with 4-bit weights, from the C3 library's entry points alone (torch holds the
memory and applies the activation):

    route -> slot plan -> quantise -> every expert's up product -> activation -> quantise
          -> every expert's down product, weighted -> sum over a token's experts

The last sum is c3_reduce_scatter over the top_k blocks of slots: choice j of token t is row
j * T + t of the products, so that each block holds one row a token. A step has no sizes that the
GPU decides, so a decoding step is captured into a graph once and replayed (`main`).

    python examples/expert_layer.py [tokens]
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from concurrent_gemm_dma_amd import _c3 as c3  # noqa: E402


def operand(x, rule=c3.C3_MX4_FLOOR, transpose=False, out=None):
    """(codes, scales) of a contiguous bf16 x [rows][cols], or of its transpose."""
    rows, cols = x.shape
    if out is None:
        sizes = c3.c3_mx4_bytes(*((cols, rows) if transpose else (rows, cols)))
        out = tuple(torch.empty(n, dtype=torch.uint8, device=x.device) for n in sizes)
    c3.c3_mx4_quantize(x, c3.C3_BF16, rows, cols, cols, transpose, rule, *out, torch.cuda.current_stream())
    return out


def weight_gradient(dy, x):
    """fp32 dy^T . x of one weight that all tokens share: [n][m] from dy [T][n] and x [T][m]. Both
    operands are quantised along the tokens; gradients by the rule that saturates nothing."""
    a, b = operand(dy, c3.C3_MX4_UP, True), operand(x, c3.C3_MX4_UP, True)
    (T, n), m = dy.shape, x.shape[1]
    out = torch.empty(n, m, device=x.device)
    c3.c3_mx4_gemm(*a, *b, out, c3.C3_F32, n, m, T, m, torch.cuda.current_stream())
    return out


class ExpertLayer:
    """up [E][F][D] and down [E][D][F] are quantised once; buffers are for T tokens."""

    def __init__(self, up, down, T, opts):
        self.E, self.F, self.D = up.shape
        self.T, self.k, self.opts = T, opts.top_k, opts
        self.up, self.down = operand(up.flatten(0, 1)), operand(down.flatten(0, 1))
        slots, dev = T * self.k, up.device
        whole = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
        half = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
        codes = lambda r, n: tuple(torch.empty(b, dtype=torch.uint8, device=dev)  # noqa: E731
                                   for b in c3.c3_mx4_bytes(r, n))
        self.idx, self.weights = whole(T, self.k), torch.empty(T, self.k, device=dev)
        self.order, self.offsets = whole(slots), whole(self.E + 1)
        self.x4, self.h4 = codes(T, self.D), codes(slots, self.F)
        self.h, self.z, self.y = half(slots, self.F), half(slots, self.D), half(T, self.D)

    def products(self, a, a_rows, b, weights, out):
        n, k = (self.F, self.D) if out is self.h else (self.D, self.F)
        c3.c3_mx4_gemm_experts(*a, a_rows, *b, self.order, self.offsets, weights, out, c3.C3_BF16, self.T, self.k,
                               self.E, n, k, n, torch.cuda.current_stream())

    def forward(self, x, logits):
        """bf16 y [T][D] of bf16 x [T][D] and fp32 logits [T][E]; a buffer of the layer's own."""
        T, k, s = self.T, self.k, torch.cuda.current_stream()
        c3.c3_route(logits, c3.C3_F32, T, self.E, self.E, self.opts, None, self.idx, self.weights, s)
        c3.c3_route_plan(self.idx, T, k, self.E, self.order, self.offsets, s)
        operand(x, out=self.x4)
        self.products(self.x4, T, self.up, None, self.h)
        torch.nn.functional.silu(self.h, inplace=True)
        operand(self.h, out=self.h4)
        self.products(self.h4, T * k, self.down, self.weights, self.z)
        c3.c3_reduce_scatter(self.y, list(self.z.view(k, T, self.D)), T * self.D * 2, None, s)
        return self.y

    def router_gradient(self, logits, dy):
        """dlogits [T][E] of the last forward, from dy [T][D]: a weight's gradient is its expert's
        unweighted output times dy."""
        each = torch.empty_like(self.z)
        self.products(self.h4, self.T * self.k, self.down, None, each)
        dw = (each.view(self.k, self.T, self.D).float() * dy.float()).sum(-1).t().contiguous()
        dlogits = torch.empty_like(logits)
        c3.c3_route_backward(logits, c3.C3_F32, self.T, self.E, self.E, self.opts, self.idx, dw, dlogits, self.E,
                             torch.cuda.current_stream())
        return dlogits


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
    dy = randn(T, D).bfloat16()
    print("router gradient", tuple(layer.router_gradient(logits, dy).shape),
          "weight gradient", tuple(weight_gradient(dy, x).shape))
    torch.cuda.synchronize()


if __name__ == "__main__":
    main(*map(int, sys.argv[1:2]))
