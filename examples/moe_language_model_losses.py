"""Training a small mixture-of-experts language-model head on the library's losses.

One step, as a training program runs it:

    router logits   gemm_bf16_nt_ordered   FP32, strict order
    routing         router_topk            weights, experts, counts, balance loss, z-loss
    experts         gemm_bf16_nt           each expert's rows
    loss            gemm_bf16_nt_xent      cross entropy over the vocabulary, no logits stored

and back: gemm_bf16_nt_xent_backward gives the hidden states' and the head's
gradients, router_topk_backward the router's.  The two operators appear as
torch.autograd functions, so the rest of the step is ordinary PyTorch.

    python examples/moe_language_model_losses.py [--steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_tcgen05_gb300 as g  # noqa: E402


class LinearCrossEntropy(torch.autograd.Function):
    """Mean cross entropy of X W^T over the rows whose target is not negative."""

    @staticmethod
    def forward(ctx, X, W, target):
        loss, lse = g.gemm_bf16_nt_xent(X, W, target)
        rows = (target >= 0).sum().clamp(min=1)
        ctx.save_for_backward(X, W, target, lse, rows)
        return loss.sum() / rows

    @staticmethod
    def backward(ctx, grad):
        X, W, target, lse, rows = ctx.saved_tensors
        dloss = (grad / rows).expand(X.shape[0]).contiguous()
        dX, dW = g.gemm_bf16_nt_xent_backward(X, W, target, lse, dloss, need_dx=ctx.needs_input_grad[0],
                                              need_dw=ctx.needs_input_grad[1])
        return dX, dW, None


class Route(torch.autograd.Function):
    """Expert weights, experts, counts and the [balance, z] losses of X Wr^T."""

    @staticmethod
    def forward(ctx, X, Wr, k, valid):
        logits = g.gemm_bf16_nt_ordered(X, Wr)
        r = g.router_topk(logits, k, valid=valid, normalize=True)
        ctx.save_for_backward(X, Wr, logits, r.experts, r.lse, r.counts)
        ctx.mark_non_differentiable(r.experts, r.counts)
        return r.weights, r.losses, r.experts, r.counts

    @staticmethod
    def backward(ctx, dweights, dlosses, _experts, _counts):
        X, Wr, logits, experts, lse, counts = ctx.saved_tensors
        d = g.router_topk_backward(logits, experts, lse, counts, dweights=dweights.contiguous(),
                                   dlosses=dlosses.contiguous(), normalize=True, dtype=torch.bfloat16)
        # E is a multiple of 8 here, as gemm_bf16_nn wants its K
        return g.gemm_bf16_nn(d, Wr), g.gemm_bf16_nn(d.T.contiguous(), X), None, None


class ExpertRows(torch.autograd.Function):
    """rows . We^T of one expert (plain products in the backward pass)."""

    @staticmethod
    def forward(ctx, rows, We):
        ctx.save_for_backward(rows, We)
        return g.gemm_bf16_nt(rows, We)

    @staticmethod
    def backward(ctx, grad):
        rows, We = ctx.saved_tensors
        return grad @ We, grad.T @ rows


def moe_layer(X, Wr, experts_w, k, valid):
    """X + sum over the chosen experts of weight * expert(X), with the routing losses and counts."""
    weights, losses, experts, counts = Route.apply(X, Wr, k, valid)
    out = X.float()
    for e, We in enumerate(experts_w):
        at = (experts == e).nonzero()          # (row, place) of the rows that chose e
        if at.numel():
            y = ExpertRows.apply(X[at[:, 0]], We)
            out = out.index_add(0, at[:, 0], y.float() * weights[at[:, 0], at[:, 1], None])
    return out.bfloat16(), losses, counts


def train(steps=60, rows=2048, hidden=256, vocab=8191, experts=16, k=2, seed=0, report=print):
    """Returns the (cross entropy, balance, z) of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std)

    # 32-bit master weights, BF16 copies for the products
    masters = [normal(experts, hidden, std=0.3)] + \
        [normal(hidden, hidden, std=hidden ** -0.5) for _ in range(experts)] + \
        [normal(vocab, hidden, std=hidden ** -0.5)]
    tokens = normal(64, hidden, std=1.0)                     # 64 kinds of token, each with its successor
    successor = torch.randint(0, vocab, (64,), generator=gen, device="cuda")
    optimiser = torch.optim.Adam(masters, lr=3e-3)
    history = []
    for step in range(steps):
        kind = torch.randint(0, 64, (rows,), generator=gen, device="cuda")
        X = (tokens[kind] + normal(rows, hidden, std=0.3)).bfloat16()
        target = successor[kind]
        valid = (torch.rand(rows, generator=gen, device="cuda") < 0.9).to(torch.uint8)
        target = torch.where(valid != 0, target, torch.full_like(target, -100))   # padding has no loss
        Wr, *We, Wv = [m.bfloat16().requires_grad_(True) for m in masters]
        Y, routing, counts = moe_layer(X, Wr, We, k, valid)
        xent = LinearCrossEntropy.apply(Y, Wv, target)
        (xent + 1e-2 * routing[0] + 1e-3 * routing[1]).backward()
        for m, w in zip(masters, [Wr, *We, Wv]):
            m.grad = w.grad.float() if w.grad is not None else torch.zeros_like(m)
        optimiser.step()
        history.append((xent.item(), routing[0].item(), routing[1].item()))
        if report and (step % 10 == 0 or step == steps - 1):
            report(f"step {step:3d}  cross entropy {history[-1][0]:7.4f}  balance {history[-1][1]:6.4f}  "
                   f"z {history[-1][2]:7.3f}  rows per expert {counts[:-1].tolist()}")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps)
