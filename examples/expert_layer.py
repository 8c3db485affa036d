"""A mixture-of-experts layer whose weights and activations are microscaled 4-bit: prompts, then decode steps from a captured
graph.

    python examples/expert_layer.py [--hidden 2048 --width 1408 --experts 64 --top 6 --tokens 4096 --step 8]

A pass is moe_plan (each token's experts, the tokens sorted by expert) -> moe_quantize (each token's row to its experts) ->
moe_gemm, gated -> moe_quantize -> moe_gemm -> moe_combine, on one stream and with no host copy in between.  Weights are
random; the passes are checked against float64 of what the quantized matrices stand for.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantized_weight_gb300 import qmm  # noqa: E402


class Layer:
    """One layer's router and experts: y = sum over a token's experts of weight * down(silu(gate(x)) * up(x))."""

    def __init__(self, hidden, width, experts, top, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.top, self.experts = top, experts
        self.router = torch.randn(hidden, experts, generator=g, device="cuda") * hidden ** -0.5

        def weights(*shape):                             # an expert at a time: float32 weights are 7 times as large
            made = [qmm.mx4_quantize(torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5) for _ in range(experts)]
            return tuple(torch.stack(t) for t in zip(*made))
        self.gate_up, self.down = weights(2, width, hidden), weights(hidden, width)

    def forward(self, x):
        """x [T, hidden], float32 or bfloat16: (y like x, and what the experts were given and gave)."""
        logits = x.float() @ self.router
        _, weights, places, starts, counts = qmm.moe_plan(logits, self.top)
        rows, routed = qmm.moe_rows(len(x), self.experts, self.top), len(x) * self.top
        h = qmm.moe_gemm(*qmm.moe_quantize(x, places, rows), *self.gate_up, starts, counts, routed=routed, gated=True,
                         dtype=x.dtype)
        y = qmm.moe_gemm(*qmm.moe_quantize(h, places, rows, sorted=True), *self.down, starts, counts, routed=routed, dtype=x.dtype)
        return qmm.moe_combine(y, weights, places), (logits, h)

    def exact(self, x, logits, h, t):
        """float64 y of token t, from the same router's logits and the same quantized matrices."""
        best = torch.topk(logits[t], self.top)
        w = torch.softmax(best.values.double(), 0)
        xq = qmm.mx4_dequant(*qmm.mx4_quantize(x[t:t + 1]))[0].double()
        y = 0
        for share, e in zip(w, best.indices):
            g, u = (qmm.mx4_dequant(self.gate_up[0][e], self.gate_up[1][e])[i].double() @ xq for i in (0, 1))
            z = (g * torch.sigmoid(g) * u).to(x.dtype)[None]           # (rounded as h is, then quantized as h is)
            z = qmm.mx4_dequant(*qmm.mx4_quantize(z))[0].double()
            y = y + share * (qmm.mx4_dequant(self.down[0][e], self.down[1][e]).double() @ z)
        return y


def run(hidden=2048, width=1408, experts=64, top=6, tokens=4096, step=8, steps=32, seed=0):
    """A prompt of bfloat16 tokens, then captured decode steps of float32.  Returns the relative error of some of the prompt's
    tokens and of the last step's, and the microseconds of both passes."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    layer = Layer(hidden, width, experts, top, seed=seed)

    def error(x, y, aux, some):
        want = torch.stack([layer.exact(x, *aux, t) for t in some])
        return float((y[some].double() - want).norm() / want.norm())

    def timed(f, n):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(n):
            f()
        end.record()
        qmm.check()
        return begin.elapsed_time(end) * 1e3 / n

    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    y, aux = layer.forward(x)
    some = sorted({0, tokens // 3, tokens // 2, tokens - 1})
    prompt_error, prompt_us = error(x, y, aux, some), timed(lambda: layer.forward(x), 5)

    x = torch.randn(step, hidden, generator=g, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x)                                 # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, aux = layer.forward(x)

    def one():
        x.copy_(torch.tanh(x + y))                       # the next tokens
        graph.replay()
    one()
    step_us = timed(one, steps)
    return prompt_error, error(x, y, aux, list(range(step))), prompt_us, step_us


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("hidden", 2048), ("width", 1408), ("experts", 64), ("top", 6), ("tokens", 4096), ("step", 8), ("steps", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    args = vars(ap.parse_args())
    prompt_error, step_error, prompt_us, step_us = run(**args)
    print(f"{args['tokens']} tokens: {prompt_us:.0f} us, relative error {prompt_error:.1e}; {args['step']} tokens: {step_us:.0f} us a "
          f"step, relative error {step_error:.1e}")


if __name__ == "__main__":
    main()
