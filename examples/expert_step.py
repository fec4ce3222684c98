"""A decode step through an adapted projection and a routed expert layer, and the adapters' training step.

    python examples/expert_step.py [--tokens T] [--steps N]

``ExpertBlock`` holds the weights (random here): a projection shared by all
requests with one low-rank adapter per request, a router, and the experts.
``step`` runs the tokens of a decode step, each with its request's adapter:

    y   = mm_lowrank_matmul(x, W, A, B, adapter)      projection + adapters
    l   = mm_matmul(y, router)                        router logits
    i,w = mm_route_topk(l, k)                         experts and weights
    out = mm_moe_layer(y, gate, up, down, i, w)       the picked experts

``adapter_gradients`` takes the gradient of y back to the adapters, for the
rows of a training batch.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_gemm_gb300 as qg  # noqa: E402


class ExpertBlock:
    def __init__(self, hidden=1024, ffn=512, experts=32, picks=4, adapters=8, rank=16, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen, device=device) * scale).to(dtype)

        self.picks = picks
        self.W = normal(hidden, hidden, scale=hidden ** -0.5)
        self.A = normal(adapters, hidden, rank, scale=hidden ** -0.5)
        self.B = normal(adapters, rank, hidden, scale=rank ** -0.5)
        self.scales = torch.full((adapters,), 0.5, device=device)
        self.router = normal(hidden, experts, scale=hidden ** -0.5)
        self.gate_up = normal(experts, hidden, 2 * ffn, scale=hidden ** -0.5)
        self.gate, self.up = self.gate_up[:, :, :ffn], self.gate_up[:, :, ffn:]     # halves of one tensor
        self.down = normal(experts, ffn, hidden, scale=ffn ** -0.5)

    def step(self, x, adapter):
        """(y, expert indices, expert weights, out) of the tokens x [T, hidden]; adapter [T], -1 for none."""
        y = qg.mm_lowrank_matmul(x, self.W, self.A, self.B, adapter, self.scales)
        indices, weights = qg.mm_route_topk(qg.mm_matmul(y, self.router), self.picks, normalize=1)
        return y, indices, weights, qg.mm_moe_layer(y, self.gate, self.up, self.down, indices, weights)

    def adapter_gradients(self, dy, x, adapter):
        """(dx, dA, dB) of the adapted projection, its shared matrix frozen."""
        return qg.mm_lowrank_matmul_grad(dy, x, self.W, self.A, self.B, adapter, self.scales)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--steps", type=int, default=100)
    args = ap.parse_args()
    block = ExpertBlock()
    x = torch.randn((args.tokens, block.W.shape[0]), device="cuda").to(block.W.dtype)
    adapter = torch.arange(args.tokens, device="cuda", dtype=torch.int32) % (block.A.shape[0] + 1) - 1
    block.step(x, adapter)                   # first call: per-device queries
    graph = torch.cuda.CUDAGraph()           # the step's launches, replayed as one
    with torch.cuda.graph(graph):
        y, indices, weights, out = block.step(x, adapter)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print("%d tokens: %.1f us a step; experts of token 0: %s, weights %s" %
          (args.tokens, start.elapsed_time(end) * 1e3 / args.steps, indices[0].tolist(),
           ["%.3f" % w for w in weights[0].tolist()]))
    dx, dA, dB = block.adapter_gradients(torch.randn_like(y), x, adapter)
    print("adapter gradients: |dA| %.4f, |dB| %.4f" % (dA.float().norm().item(), dB.float().norm().item()))
    assert qg.mm_get_device_status() == "MM_OK"


if __name__ == "__main__":
    main()
