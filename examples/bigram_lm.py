"""Trains a small residual MLP language model with the operators, then scores
tokens one at a time with the same weights, as a server would.

    python examples/bigram_lm.py [--steps 60] [--batch 2048] [--hidden 512] [--vocab 5003] [--layers 2] [--dtype bf16]

The model predicts the next token from the current one:
    h = embedding[token]                                     (fp32 residual stream)
    h, x = norm_residual(h, y)   z, a = linear(x, w1, gelu)   y = linear(a, w2)      for each layer
    h, x = norm_residual(h, y)   loss = linear_xent(x, vocabulary, next token)
The data is a synthetic Markov chain, so the loss a perfect model reaches is
known.  Every step runs the gradient of each operator and updates fp32 master
weights; nothing here uses autograd.
"""
import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import dense_gemm_elementwise_amd as ge  # noqa: E402

BRANCH = 4  # every token is followed by one of this many, evenly


class Model:
    """Weights (16-bit, with fp32 masters) and the forward and backward over the operators."""

    def __init__(self, vocab, hidden, layers, dtype, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(shape, generator=g, device=device) * std
        self.layers, self.dtype = layers, dtype
        m = {"embedding": normal(vocab, hidden, std=0.5), "vocabulary": normal(vocab, hidden, std=hidden ** -0.5)}
        for i in range(layers):
            m[f"w1.{i}"] = normal(4 * hidden, hidden, std=hidden ** -0.5)
            m[f"b1.{i}"] = torch.zeros(4 * hidden, device=device)
            m[f"w2.{i}"] = normal(hidden, 4 * hidden, std=0.5 * hidden ** -0.5)
        for i in range(layers + 1):
            m[f"pre.{i}"] = torch.ones(hidden, device=device)
            m[f"post.{i}"] = torch.ones(hidden, device=device)
        self.master = m
        self.moment = {k: torch.zeros_like(v) for k, v in m.items()}
        self.square = {k: torch.zeros_like(v) for k, v in m.items()}
        self.round()

    def round(self):
        self.w = {k: v.to(self.dtype) for k, v in self.master.items()}

    def forward(self, tokens, save=None):
        """The normalised last hidden rows; `save` collects what the backward needs."""
        w = self.w
        h = self.master["embedding"][tokens]
        y = torch.zeros(h.shape, dtype=self.dtype, device=h.device)
        for i in range(self.layers):
            h, x = ge.norm_residual(h, y, w_post=w[f"post.{i}"], w_pre=w[f"pre.{i}"])
            if save is None:
                a = ge.linear(x, w[f"w1.{i}"], w[f"b1.{i}"], act="gelu")
            else:
                a, z = ge.linear(x, w[f"w1.{i}"], w[f"b1.{i}"], act="gelu", save_z=True)
                save.append((h, y, x, z, a))
            y = ge.linear(a, w[f"w2.{i}"])
        h, x = ge.norm_residual(h, y, w_post=w[f"post.{self.layers}"], w_pre=w[f"pre.{self.layers}"])
        if save is not None:
            save.append((h, y, x))
        return x

    def gradients(self, tokens, target):
        """(mean loss, gradients by name)"""
        w, saved, grads = self.w, [], {}
        x = self.forward(tokens, saved)
        loss, lse = ge.linear_xent(x, w["vocabulary"], target)
        dloss = torch.full_like(loss, 1.0 / loss.numel())
        dx, grads["vocabulary"] = ge.linear_xent_backward(dloss, x, w["vocabulary"], target, lse)
        h, y, _ = saved[-1]
        dh = torch.zeros_like(h)
        for i in range(self.layers, -1, -1):
            dh, dy, grads[f"post.{i}"], grads[f"pre.{i}"], _ = ge.norm_residual_backward(
                dx, dh, h, y, w_post=w[f"post.{i}"], w_pre=w[f"pre.{i}"])
            if i == 0:
                break
            h, y, x, z, a = saved[i - 1]
            da, grads[f"w2.{i - 1}"], _ = ge.linear_backward(dy, a, w[f"w2.{i - 1}"], need_dbias=False)
            dx, grads[f"w1.{i - 1}"], grads[f"b1.{i - 1}"] = ge.linear_backward(da, x, w[f"w1.{i - 1}"], z, act="gelu")
        grads["embedding"] = torch.zeros_like(self.master["embedding"]).index_add_(0, tokens, dh)
        return loss.mean(), grads

    def update(self, grads, step, lr=3e-3, b1=0.9, b2=0.99):
        for k, g in grads.items():
            g = g.float()
            self.moment[k].lerp_(g, 1 - b1)
            self.square[k].lerp_(g * g, 1 - b2)
            m, s = self.moment[k] / (1 - b1 ** step), self.square[k] / (1 - b2 ** step)
            self.master[k].sub_(lr * m / (s.sqrt() + 1e-8))
        self.round()

    def score(self, token, target):
        """The log probability of one next token: the single-row calls."""
        loss, _ = ge.linear_xent(self.forward(token), self.w["vocabulary"], target)
        return -loss


def batch(successors, n, generator):
    vocab = successors.shape[0]
    tokens = torch.randint(0, vocab, (n,), generator=generator, device=successors.device)
    pick = torch.randint(0, BRANCH, (n,), generator=generator, device=successors.device)
    return tokens, successors[tokens, pick]


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--batch", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=5003)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--dtype", choices=("bf16", "f16"), default="bf16")
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)
    successors = torch.randint(0, a.vocab, (a.vocab, BRANCH), generator=g, device=dev)
    model = Model(a.vocab, a.hidden, a.layers, {"bf16": torch.bfloat16, "f16": torch.float16}[a.dtype], dev)
    losses = []
    for step in range(1, a.steps + 1):
        tokens, target = batch(successors, a.batch, g)
        loss, grads = model.gradients(tokens, target)
        model.update(grads, step)
        losses.append(loss.item())
        if step == 1 or step % 10 == 0:
            print(f"step {step}: loss {losses[-1]:.4f} (uniform {math.log(a.vocab):.4f}, best {math.log(BRANCH):.4f})",
                  flush=True)
    tokens, target = batch(successors, 8, g)
    rows, _ = ge.linear_xent(model.forward(tokens), model.w["vocabulary"], target)
    single = torch.cat([model.score(tokens[i:i + 1], target[i:i + 1]) for i in range(8)])
    gap = (rows + single).abs().max().item()
    print(f"8 tokens scored one at a time: largest difference from the batch {gap:.5f}", flush=True)
    return losses, gap


if __name__ == "__main__":
    main()
