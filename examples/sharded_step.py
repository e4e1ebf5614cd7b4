"""Training steps over sharded parameters, with every collective and operator of the library in its place.

    python examples/sharded_step.py [--steps 60]

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
    E, W = 0, 1  # the group's parameters

    def __init__(self, R: int, vocab: int, dim: int, tokens: int, seed: int = 0):
        self.R, self.vocab, self.dim, self.tokens = R, vocab, dim, tokens
        self.group = tide.Group(R, [(vocab, dim), (dim, dim)])
        S = self.group.S
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.master = torch.zeros(R, S, device="cuda")
        for k, view in enumerate(self.group.pieces(self.master)):  # rank by rank, E before W
            view.normal_(0.0, 0.02 if k % 2 == self.E else dim ** -0.5, generator=g)
        self.shards = self.master.bfloat16()
        self.grads, self.exp_avg, self.exp_avg_sq = (torch.zeros(R, S, device="cuda") for _ in range(3))
        pieces = [self.group.pieces(b) for b in (self.master, self.grads, self.exp_avg, self.exp_avg_sq, self.shards)]
        self.list = tide.TensorList([x.numel() for x in pieces[0]])
        # buffers that every step passes again are marshalled once
        self.tables = [tide.pointer_table(xs) for xs in pieces]
        self.workspace = self.group.embedding_grad_workspace(self.E, R * tokens)
        self.params = [torch.empty(n, dim, dtype=torch.bfloat16, device="cuda") for n in (vocab, dim)]
        self.norm = torch.zeros(1, device="cuda")
        self.count = 0

    def step(self, batches, lr: float = 3e-3, max_norm: float = 1.0, weight_decay: float = 0.01) -> torch.Tensor:
        """One step on R (tokens, targets) pairs; returns the mean loss over the ranks."""
        R, scale = self.R, self.dim ** 0.5
        self.group.all_gather(list(self.shards), [p.view(-1) for p in self.params])
        dense, ids, douts, total = [], [], [], 0.0
        for tokens, targets in batches:
            x = torch.empty(tokens.numel(), self.dim, dtype=torch.bfloat16, device="cuda")
            self.group.embedding(self.E, list(self.shards), tokens, x, scale)
            x.requires_grad_(True)
            E, W = (p.detach().requires_grad_(True) for p in self.params)
            logits = torch.relu(x @ W) @ E.t()
            loss = torch.nn.functional.cross_entropy(logits.float(), targets) / R  # the shards hold sums over the ranks
            loss.backward()
            dense.append([E.grad.contiguous().view(-1), W.grad.contiguous().view(-1)])
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
    a = ap.parse_args()
    model = ShardedModel(a.ranks, a.vocab, a.dim, a.tokens)
    for step in range(a.steps):
        loss = model.step(batches(a.ranks, a.vocab, a.tokens, step))
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:4d}  loss {float(loss):.4f}  gradient norm {float(model.norm):.4f}")


if __name__ == "__main__":
    main()
