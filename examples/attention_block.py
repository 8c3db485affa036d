"""An attention block whose weights and whose key/value cache are both 4-bit: prompts in one step, then decode steps
from a captured graph.

    python examples/attention_block.py [--hidden 2048 --heads 16 --kv-heads 8 --head-dim 128 --requests 8 --prompt 500]

A step is kv_plan (slots, positions, block tables) -> the fused q/k/v product (gemm for prompts, gemv for decode) ->
rotary positions -> kv_append -> kv_attend -> the output product, all on one stream and with no host copy in between.
Weights are random; the last step is checked against float64 over what kv_read gives back.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantized_weight_gb300 import qmm  # noqa: E402

GROUP = 64


class Block:
    """One block's weights and cache, and the requests that it serves (at most 8: a decode product's tokens)."""

    def __init__(self, hidden, heads, kv_heads, head_dim, requests, max_len, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.D, self.page, self.B = heads, kv_heads, head_dim, page, requests
        self.n_qkv, self.n_out = (heads + 2 * kv_heads) * head_dim, hidden
        self.w_qkv = qmm.quantize(torch.randn(self.n_qkv, hidden, generator=g, device="cuda") * hidden ** -0.5, GROUP)
        self.w_out = qmm.quantize(torch.randn(hidden, heads * head_dim, generator=g, device="cuda") * hidden ** -0.5, GROUP)
        blocks = -(-max_len // page)
        self.cache = qmm.kv_cache(requests * blocks, kv_heads, head_dim, page, GROUP)
        self.table = torch.full((requests, blocks), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(requests * blocks, generator=g, device="cuda").int()   # the serving loop's free list
        self.cached = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.freqs = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda") / head_dim)

    def rotate(self, x, positions):
        """Rotary positions of x [T, heads, D], first half against second half."""
        a = positions[:, None, None] * self.freqs
        c, s = a.cos(), a.sin()
        lo, hi = x.float().chunk(2, -1)
        return torch.cat((lo * c - hi * s, hi * c + lo * s), -1).to(x.dtype)

    def step(self, x, fresh, max_fresh, workspace):
        """x [T, hidden] of the requests' new tokens, one request after the other: the block's output [T, hidden].
        bfloat16 x goes through the prompt products, float32 x (T <= 8) through the decode products."""
        product = qmm.gemm if x.dtype is torch.bfloat16 else qmm.gemv
        T, H, K, D = len(x), self.heads, self.kv_heads, self.D
        slots, positions, cu, lens, need = qmm.kv_plan(self.cached, fresh, self.free, self.table, T, self.page)
        qkv = product(x, *self.w_qkv, self.n_qkv, 4, GROUP).to(x.dtype).view(T, H + 2 * K, D)
        qk = self.rotate(qkv[:, :H + K], positions)
        qmm.kv_append(qk[:, H:], qkv[:, H + K:], slots, self.cache, self.page, GROUP)
        y = qmm.kv_attend(qk[:, :H], self.cache, self.table, lens, self.page, GROUP, workspace, cu=cu, max_fresh=max_fresh)
        out = product(y.view(T, H * D), *self.w_out, self.n_out, 4, GROUP)
        self.cached.copy_(lens)
        # a serving loop takes the pages off its list; here the list turns by as many
        at = torch.arange(len(self.free), device="cuda")
        self.free.copy_(self.free[(at + need) % len(self.free)])
        return out, qk[:, :H], y

    def exact(self, q):
        """Attention of one query a request [B, heads, D] over everything that its request has cached, in float64."""
        outs = []
        for b in range(self.B):
            n = int(self.cached[b])
            j = torch.arange(n, device="cuda")
            slots = (self.table[b, j // self.page] * self.page + j % self.page).int()
            k, v = (t.double().repeat_interleave(self.heads // self.kv_heads, 1)
                    for t in qmm.kv_read(slots, self.cache, self.D, self.page, GROUP))
            p = torch.softmax(torch.einsum("hd,nhd->hn", q[b].double(), k) * self.D ** -0.5, -1)
            outs.append(torch.einsum("hn,nhd->hd", p, v))
        return torch.stack(outs)


def run(hidden=2048, heads=16, kv_heads=8, head_dim=128, requests=8, prompt=500, steps=32, seed=0):
    """Prompts of ragged lengths up to `prompt`, then `steps` decode steps.  Returns the relative error of the prompt's last
    queries and of the last decode step, the microseconds of a decode step, and the block."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    block = Block(hidden, heads, kv_heads, head_dim, requests, prompt + steps + 1, seed=seed)
    lens = [max(1, prompt - 37 * b) for b in range(requests)]
    fresh = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = qmm.kv_attend_workspace(requests, heads, kv_heads, head_dim, max(lens))
    x = torch.randn(sum(lens), hidden, generator=g, device="cuda").bfloat16()
    _, q, y = block.step(x, fresh, max(lens), ws)
    qmm.check()
    last = torch.tensor(lens).cumsum(0).cuda() - 1

    def error(q, y):
        want = block.exact(q)
        return float((y.double() - want).norm() / want.norm())
    errors = [error(q[last], y[last])]

    x = torch.randn(requests, hidden, generator=g, device="cuda")
    one = torch.ones(requests, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, one, 1, ws)                          # warm-up, a step like the others
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, q, y = block.step(x, one, 1, ws)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(steps):
        graph.replay()
        x.copy_(torch.tanh(out))                           # the next tokens
    end.record()
    qmm.check()
    errors.append(error(q, y))
    return errors[0], errors[1], begin.elapsed_time(end) * 1e3 / steps, block


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("hidden", 2048), ("heads", 16), ("kv-heads", 8), ("head-dim", 128), ("requests", 8), ("prompt", 500),
                        ("steps", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    args = vars(ap.parse_args())
    prompt_error, decode_error, us, block = run(**args)
    print(f"prompts: relative error {prompt_error:.1e}; decode: {us:.0f} us a step, relative error {decode_error:.1e}; "
          f"cache {block.cache.numel() / 1e6:.1f} MB ({block.cache.numel() * 8 / (block.cache.shape[0] * block.page * block.kv_heads * 2 * block.D):.1f} bits a value)")


if __name__ == "__main__":
    main()
