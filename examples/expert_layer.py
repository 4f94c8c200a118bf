"""A feed-forward layer of routed experts in e4m3, as a serving program would
run it on one GPU:

    router scores -> the two best experts of each token -> rows in expert order
    ox_quantize_fp8(index)    gather and quantise the tokens
    ox_gemm_grouped_fp8       expand, bias and GELU
    ox_quantize_fp8           quantise the hidden rows
    ox_gemm_grouped_fp8       project back
    weighted sum of each token's two rows

Nothing is read back to the host between the steps, so the layer is also
recorded into a HIP graph and replayed.  Prints the time of both and how far
the result is from the same layer in fp32.

    python examples/expert_layer.py [--tokens 64] [--experts 8] [--width 1024] [--hidden 4096]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv_implicit_gemm_amd as ox  # noqa: E402

F8 = torch.float8_e4m3fn
TOP = 2


class ExpertLayer:
    def __init__(self, tokens, experts, width, hidden, generator):
        def normal(*shape):
            return torch.randn(shape, generator=generator, device="cuda")
        self.E = experts
        self.router = normal(width, experts) * width ** -0.5
        self.W1 = (normal(experts, hidden, width) * width ** -0.5).bfloat16()
        self.W2 = (normal(experts, width, hidden) * hidden ** -0.5).bfloat16()
        self.b1 = (0.1 * normal(experts, hidden)).bfloat16()
        self.q1, self.s1 = self.quantise(self.W1)
        self.q2, self.s2 = self.quantise(self.W2)
        rows = tokens * TOP
        blocks = lambda n: (n + 127) // 128                                    # noqa: E731
        self.xq = torch.empty(rows, width, dtype=F8, device="cuda")
        self.xs = torch.empty(blocks(width), rows, device="cuda")
        self.h = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda")
        self.hq = torch.empty(rows, hidden, dtype=F8, device="cuda")
        self.hs = torch.empty(blocks(hidden), rows, device="cuda")
        self.y = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")

    @staticmethod
    def quantise(W):
        parts = [ox.ox_quantize_fp8(w, block_rows=128) for w in W]
        return torch.stack([q.view(torch.uint8) for q, _ in parts]).view(F8), torch.stack([s for _, s in parts])

    def route(self, X):
        """Weights [tokens, TOP], and for the rows in expert order: their token,
        their place in that order, and the experts' offsets."""
        weight, expert = torch.softmax(X.float() @ self.router, dim=1).topk(TOP, dim=1)
        weight = weight / weight.sum(dim=1, keepdim=True)
        expert = expert.reshape(-1)
        order = torch.argsort(expert, stable=True)
        place = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device="cuda"))
        counts = (expert.unsqueeze(1) == torch.arange(self.E, device="cuda")).sum(dim=0, dtype=torch.int32)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0, dtype=torch.int32)])
        return weight, (order // TOP).to(torch.int32), place, offsets

    def __call__(self, X):
        weight, token, place, offsets = self.route(X)
        ox.ox_quantize_fp8(X, index=token, Q=self.xq, scales=self.xs)
        ox.ox_gemm_grouped_fp8(self.xq, self.xs, self.q1, self.s1, offsets, bias=self.b1, act="gelu", Y=self.h)
        ox.ox_quantize_fp8(self.h, Q=self.hq, scales=self.hs)
        ox.ox_gemm_grouped_fp8(self.hq, self.hs, self.q2, self.s2, offsets, Y=self.y)
        rows = self.y[place].view(X.shape[0], TOP, -1).float()
        return (rows * weight.unsqueeze(2)).sum(dim=1).to(X.dtype)

    def in_fp32(self, X):
        weight, token, place, offsets = self.route(X)
        rows, at = X.float()[token.long()], offsets.tolist()
        out = torch.empty(rows.shape[0], self.W2.shape[1], device="cuda")
        for e in range(self.E):
            h = rows[at[e]:at[e + 1]] @ self.W1[e].float().t() + self.b1[e].float()
            out[at[e]:at[e + 1]] = torch.nn.functional.gelu(h) @ self.W2[e].float().t()
        return (out[place].view(X.shape[0], TOP, -1) * weight.unsqueeze(2)).sum(dim=1)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 64), ("experts", 8), ("width", 1024), ("hidden", 4096)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = ExpertLayer(a.tokens, a.experts, a.width, a.hidden, g)
    X = torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16()
    out = layer(X)
    want = layer.in_fp32(X)
    off = ((out.float() - want).norm() / want.norm()).item()

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(X)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        captured = layer(X)
    graph.replay()
    torch.cuda.synchronize()
    same = torch.equal(captured, out)

    def clock(f, n=50):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e6
    print("%d tokens, %d experts of %d x %d: eager %.1f us, graph %.1f us, %.2f%% off fp32, replay %s" % (
        a.tokens, a.experts, a.hidden, a.width, clock(lambda: layer(X)), clock(graph.replay), 100 * off,
        "equal" if same else "DIFFERENT"))
    return off, same


if __name__ == "__main__":
    main()
