"""Training steps over sharded parameters, with every collective and operator of the library in its place.

    python examples/sharded_step.py [--steps 60] [--experts 8 --choices 2]

A small language model whose output layer shares the embedding table:

    x = sqrt(D) * E[token],   h = relu(x @ W),   logits = h @ E^T

R ranks (buffers on one GPU) hold E and W as packed bf16 shards with fp32 masters.  Each rank has its own
batch of tokens.  One step is

    all_gather       the ranks' bf16 shards -> E and W, for the matrix products
    embedding        every rank's rows of E, straight from the shards
    (matrix products and their gradients: PyTorch)
    reduce_scatter   the ranks' dense bf16 gradients of E (output layer) and W -> fp32 shards
    embedding_grad   the lookup's gradients of all ranks, added to E's pieces of those shards
    grad_norm, adamw the norm over all pieces, the clipped step, the next bf16 shards

With --experts the hidden layer is one of experts, a matrix W_e and a row of the router G each:

    p = softmax of the k largest of x @ G^T,   h = sum over these of p_e * relu(x @ W_e^T)

whose matrices go from the shards to 8 bits (all_gather_fp8, beside the all_gather of E and G), whose rows go to their experts and back
(sort, dispatch_fp8, combine), and whose products and gradients are formed in 8 bits (matmul, quantize, weight_grad).

The text is a fixed cycle through the vocabulary, so the next token can be learnt.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import all_gather_tide_gb300 as tide  # noqa: E402


class ShardedModel:
    E, W = 0, 1  # the group's parameters; with experts G, the router, in W's place, and their matrices behind it

    def __init__(self, R: int, vocab: int, dim: int, tokens: int, seed: int = 0, experts: int = 0, choices: int = 2):
        self.R, self.vocab, self.dim, self.tokens, self.experts = R, vocab, dim, tokens, experts
        shapes = [(vocab, dim), (experts or dim, dim)] + [(dim, dim)] * experts
        self.group = tide.Group(R, shapes)
        S = self.group.S
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.master = torch.zeros(R, S, device="cuda")
        for k, view in enumerate(self.group.pieces(self.master)):  # rank by rank, E before W
            view.normal_(0.0, 0.02 if k % len(shapes) == self.E else dim ** -0.5, generator=g)
        self.shards = self.master.bfloat16()
        self.grads, self.exp_avg, self.exp_avg_sq = (torch.zeros(R, S, device="cuda") for _ in range(3))
        pieces = [self.group.pieces(b) for b in (self.master, self.grads, self.exp_avg, self.exp_avg_sq, self.shards)]
        self.list = tide.TensorList([x.numel() for x in pieces[0]])
        # buffers that every step passes again are marshalled once
        self.tables = [tide.pointer_table(xs) for xs in pieces]
        self.workspace = self.group.embedding_grad_workspace(self.E, R * tokens)
        self.params = [torch.empty(n, dim, dtype=torch.bfloat16, device="cuda") for n, _ in shapes]
        self.norm = torch.zeros(1, device="cuda")
        self.count = 0
        if experts:
            M = tokens * choices
            self.layer = tide.Experts(experts, choices)
            self.route = self.layer.route(tokens)
            self.weights8 = tide.Fp8Weights(experts, dim, dim, transposed=True)
            self.rows8, self.dy8 = tide.Fp8Rows(M, dim), tide.Fp8Rows(M, dim)
            self.xt8, self.dyt8 = tide.Fp8Columns(M, dim, experts), tide.Fp8Columns(M, dim, experts)
            # the experts' own matrices are needed in 8 bits alone: all_gather is for a group of the others
            self.dense = tide.Group(R, shapes[:2])

    def gather(self) -> None:
        """The parameters out of the ranks' shards."""
        if not self.experts:
            self.group.all_gather(list(self.shards), [p.view(-1) for p in self.params])
            return
        # E and G come first in the shards, in the same places as in a group of their own
        self.dense.all_gather([s[:self.dense.S] for s in self.shards], [p.view(-1) for p in self.params[:2]])
        self.group.all_gather_fp8(range(2, 2 + self.experts), list(self.shards), self.weights8)

    def expert_layer(self, x, G):
        """h of tokens x and router G, and what takes h's gradient to x's, G's and the matrices'."""
        layer, route, T, dim = self.layer, self.route, x.shape[0], self.dim
        score, ids = (x.float() @ G.float().t()).topk(layer.k, dim=1)
        p = torch.softmax(score, 1)
        weights = p.detach().contiguous()
        y, h = torch.zeros(route.M, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(T, dim, dtype=torch.bfloat16, device="cuda")
        layer.sort(ids, route)
        layer.dispatch_fp8(x.detach(), route, self.rows8)
        layer.matmul(self.rows8, self.weights8, route, y)
        rows = torch.relu(y)
        layer.combine(rows, route, h, weights)

        def backward(dh):
            drows, dweights = torch.zeros_like(rows), torch.empty_like(weights)
            layer.combine_grad(dh.contiguous(), rows, route, weights, drows, dweights)
            dy = drows * (y > 0)
            layer.quantize(dy, route, rows=self.dy8, columns=self.dyt8)
            layer.quantize(x.detach(), route, columns=self.xt8, gather=True)
            dx_rows, dx = torch.empty_like(y), torch.empty_like(x)
            layer.matmul(self.dy8, self.weights8, route, dx_rows, transposed=True)
            layer.combine(dx_rows, route, dx)
            grads = [torch.empty(dim * dim, dtype=torch.bfloat16, device="cuda") for _ in range(self.experts)]
            layer.weight_grad(self.dyt8, self.xt8, route, grads)
            p.backward(dweights)  # the router's part of x's gradient, and G's
            x.grad += dx
            return grads

        return h, backward

    def step(self, batches, lr: float = 3e-3, max_norm: float = 1.0, weight_decay: float = 0.01) -> torch.Tensor:
        """One step on R (tokens, targets) pairs; returns the mean loss over the ranks."""
        R, scale = self.R, self.dim ** 0.5
        self.gather()
        dense, ids, douts, total = [], [], [], 0.0
        for tokens, targets in batches:
            x = torch.empty(tokens.numel(), self.dim, dtype=torch.bfloat16, device="cuda")
            self.group.embedding(self.E, list(self.shards), tokens, x, scale)
            x.requires_grad_(True)
            E, W = (p.detach().requires_grad_(True) for p in self.params[:2])
            h, backward = self.expert_layer(x, W) if self.experts else (torch.relu(x @ W), None)
            if backward:
                h.requires_grad_(True)
            logits = h @ E.t()
            loss = torch.nn.functional.cross_entropy(logits.float(), targets) / R  # the shards hold sums over the ranks
            loss.backward()
            grads = backward(h.grad) if backward else []
            dense.append([E.grad.contiguous().view(-1), W.grad.contiguous().view(-1), *grads])
            ids.append(tokens)
            douts.append(x.grad)
            total = total + loss.detach()
        self.group.reduce_scatter(dense, list(self.grads))
        self.group.embedding_grad(self.E, ids, douts, list(self.grads), scale, accumulate=True, workspace=self.workspace)
        master, grads, exp_avg, exp_avg_sq, shards = self.tables
        self.list.grad_norm(grads, self.norm)
        self.count += 1
        self.list.adamw(master, grads, exp_avg, exp_avg_sq, shards, lr=lr, betas=(0.9, 0.95), weight_decay=weight_decay, step=self.count,
                        norm=self.norm, max_norm=max_norm, flags=tide.TIDE_ADAMW_SKIP_NONFINITE)
        return total


def batches(R: int, vocab: int, tokens: int, step: int):
    """R pieces of a text that steps through the vocabulary."""
    out = []
    for r in range(R):
        t = (torch.arange(tokens + 1, device="cuda") * 7 + 31 * r + 101 * step) % vocab
        out.append((t[:-1].contiguous(), t[1:].contiguous()))
    return out


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=1003)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--experts", type=int, default=0)
    ap.add_argument("--choices", type=int, default=2)
    a = ap.parse_args()
    model = ShardedModel(a.ranks, a.vocab, a.dim, a.tokens, experts=a.experts, choices=a.choices)
    for step in range(a.steps):
        loss = model.step(batches(a.ranks, a.vocab, a.tokens, step))
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:4d}  loss {float(loss):.4f}  gradient norm {float(model.norm):.4f}")


if __name__ == "__main__":
    main()
