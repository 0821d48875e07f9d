"""Trains a small language model with FP4 experts on a synthetic next-token task.

    python examples/train_experts.py [--steps 60]

    x = Emb[token]                                   bfloat16
    e, p = the router's two best experts of a token and their softmax weights
    h_e = relu(Up_e x),  y = x + sum p_e * Down_e h_e    experts' products, FP4
    loss = cross entropy of y Head against the next token, without the logits

Dispatch takes the tokens' rows to their experts, combine brings them back. The
backward is written out with the same calls (dgrad and wgrad of the experts, the
gradients of combine, dispatch, the head loss and the embedding), the gradients are
clipped by their global norm and the weights updated by Adam in float32. The text is a fixed permutation of the
vocabulary: each token has one successor, so the loss can fall to zero.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_linear_layer_amd as ql  # noqa: E402


class Model:
    """Float32 weights; every step works on bfloat16 copies of them."""

    def __init__(self, vocab=512, hidden=256, inner=512, experts=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, std=0.05):
            return torch.randn(shape, generator=g, device="cuda") * std

        self.w = dict(emb=weight(vocab, hidden, std=1.0), router=weight(hidden, experts),
                      up=weight(experts, hidden, inner), down=weight(experts, inner, hidden),
                      head=weight(hidden, vocab))
        self.mean = {k: torch.zeros_like(v) for k, v in self.w.items()}
        self.var = {k: torch.zeros_like(v) for k, v in self.w.items()}
        self.t = 0

    def loss_and_grads(self, tokens, targets):
        """(mean loss, gradients by name) of one batch of tokens and next tokens."""
        w = {k: v.bfloat16() for k, v in self.w.items()}
        experts = w["up"].shape[0]
        x = ql.embed(w["emb"], tokens)
        prob = (x.float() @ self.w["router"]).softmax(1)
        weight, expert = prob.topk(2, dim=1)
        # the rows by expert; the ends of the experts' rows stay on the GPU
        xs, row_end, slot_row = ql.experts_dispatch(x, expert.to(torch.int32), experts)

        u = ql.experts_forward_mx(xs, w["up"], row_end)
        h = u.relu().bfloat16()
        d = ql.experts_forward_mx(h, w["down"], row_end)
        y = ql.experts_combine(d, slot_row, row_end, weight, x)
        loss, lse = ql.head_loss(y, w["head"], targets)

        counted = (targets >= 0).sum()
        dloss = torch.full_like(loss, 1.0) / counted
        dy, dhead = ql.head_loss_backward(y, w["head"], targets, lse, dloss)
        dd, dweight = ql.experts_combine_backward(dy, d, slot_row, row_end, weight)
        ddown = ql.experts_wgrad_mx(h, dd, row_end)
        dh = ql.experts_dgrad_mx(dd, w["down"], row_end)
        du = torch.where(u > 0, dh, 0.0).bfloat16()
        dup = ql.experts_wgrad_mx(xs, du, row_end)
        dxs = ql.experts_dgrad_mx(du, w["up"], row_end)
        # the router through the weights of the chosen experts
        dprob = torch.zeros_like(prob).scatter_(1, expert, dweight)
        dlogits = prob * (dprob - (dprob * prob).sum(1, keepdim=True))
        dx = dy.float() + ql.experts_combine(dxs, slot_row, row_end) + dlogits @ self.w["router"].t()
        demb = ql.embed_backward(dx, tokens, w["emb"].shape[0])
        grads = dict(emb=demb, router=x.float().t() @ dlogits, up=dup, down=ddown, head=dhead.float())
        return loss.sum() / counted, grads

    def step(self, tokens, targets, rate=3e-3, max_norm=1.0):
        """One training step; returns (loss, gradient norm), both on the GPU."""
        loss, grads = self.loss_and_grads(tokens, targets)
        norm = ql.clip_grads(list(grads.values()), max_norm)
        self.t += 1
        for k, g in grads.items():
            self.mean[k].lerp_(g, 0.1)
            self.var[k].lerp_(g * g, 0.01)
            m = self.mean[k] / (1 - 0.9 ** self.t)
            v = self.var[k] / (1 - 0.99 ** self.t)
            self.w[k] -= rate * m / (v.sqrt() + 1e-8)
        return loss, norm


def batch(successor, tokens, generator):
    """Random tokens and their successors; every tenth row carries no loss."""
    t = torch.randint(0, successor.numel(), (tokens,), generator=generator, device="cuda",
                      dtype=torch.int32)
    target = successor[t.long()]
    target[::10] = -1
    return t, target


def train(steps=60, tokens=2048, vocab=512, seed=0, log=print):
    g = torch.Generator(device="cuda").manual_seed(seed)
    successor = torch.randperm(vocab, generator=g, device="cuda").to(torch.int32)
    model = Model(vocab=vocab, seed=seed)
    losses = []
    for i in range(steps):
        loss, norm = model.step(*batch(successor, tokens, g))
        losses.append(float(loss))
        if i % 10 == 0 or i == steps - 1:
            log(f"step {i:4d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.3f}")
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=60)
    train(p.parse_args().steps)
