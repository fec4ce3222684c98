"""A training step of a routed expert layer, and the layer served in 8 bits.

    python examples/train_and_serve.py [--tokens T] [--steps N]

``ExpertLayer`` holds a router in fp32 and one projection per expert (random
here).  A training step calls

    l      = mm_matmul(x, router)                     router logits
    i, w   = mm_route_topk(l, k)                      experts and weights
    L, c   = mm_route_balance(l, i)                   balance loss, picks per expert
    dl     = mm_route_balance_grad(l, c, ..., base=mm_route_topk_grad(l, i, dw))
    update = mm_orthogonalize(gradients)              of the router and of all experts at once

and ``serve`` turns the experts' weights into int8 with a scale per output channel;
tokens are quantised with a scale each and multiplied:

    q, s   = mm_quantize_rows(x)
    y      = mm_int8_matmul(q, w_int8, s, w_scale)
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_gemm_gb300 as qg  # noqa: E402


class ExpertLayer:
    def __init__(self, hidden=1024, ffn=512, experts=32, picks=4, dtype=torch.bfloat16, seed=0, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.picks = picks
        self.router = torch.randn((hidden, experts), generator=gen, device=device) * hidden ** -0.5
        self.experts = (torch.randn((experts, hidden, ffn), generator=gen, device=device) * hidden ** -0.5).to(dtype)

    def route(self, x):
        """(logits, expert indices, weights) of the tokens x [T, hidden] in fp32."""
        logits = qg.mm_matmul(x, self.router)
        return (logits, *qg.mm_route_topk(logits, self.picks, normalize=1))

    def router_gradient(self, logits, indices, grad_weights, balance=0.01):
        """(balance loss, picks per expert, gradient of the logits): the gradient through the picks' weights and
        ``balance`` times the balance loss's."""
        loss, counts, _ = qg.mm_route_balance(logits, indices)
        through = qg.mm_route_topk_grad(logits, indices, grad_weights, normalize=1)
        scale = torch.full((1,), balance, device=logits.device)
        return loss, counts, qg.mm_route_balance_grad(logits, counts, scale, base=through)

    def update(self, x, grad_logits, grad_experts, rate=0.02):
        """One step along the orthogonalised gradients; the experts' are one stack [G, hidden, ffn]."""
        self.router -= rate * qg.mm_orthogonalize(qg.mm_matmul(x.t(), grad_logits))
        self.experts -= rate * qg.mm_orthogonalize(grad_experts)

    def serve(self):
        """A function (x [T, hidden], expert) -> x @ experts[expert] in 8 bits."""
        stored = [qg.mm_quantize_rows(w.t()) for w in self.experts]      # [ffn, hidden] rows: a scale per channel

        def project(x, expert):
            q, s = qg.mm_quantize_rows(x)
            w, ws = stored[expert]
            return qg.mm_int8_matmul(q, w.t(), s, ws, dtype=x.dtype)
        return project


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    block = ExpertLayer()
    x = torch.randn((args.tokens, block.router.shape[0]), device="cuda")
    dw = torch.randn((args.tokens, block.picks), device="cuda") / args.tokens
    grads = torch.randn(block.experts.shape, device="cuda").to(block.experts.dtype)

    def step():
        logits, indices, _ = block.route(x)
        loss, counts, dlogits = block.router_gradient(logits, indices, dw)
        block.update(x, dlogits, grads, rate=1e-3)
        return loss, counts

    step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(args.steps):
        loss, counts = step()
    end.record()
    torch.cuda.synchronize()
    y = block.serve()(x[:16].to(block.experts.dtype), 0)
    print("%d tokens: %.1f us a step; balance loss %.4f, most picks of an expert %d; served %s %s" %
          (args.tokens, start.elapsed_time(end) * 1e3 / args.steps, loss.item(), counts[:-1].max().item(),
           tuple(y.shape), y.dtype))


if __name__ == "__main__":
    main()
