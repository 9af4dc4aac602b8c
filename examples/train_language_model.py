"""One worker's training of a small next-token model with this library's steps.

    python examples/train_language_model.py [--steps 60] [--vocab 4096] [--dim 256] [--density 0.01]
                                            [--norm] [--distill]

Each step looks the tokens' rows up in an embedding table (``embedding_lookup``),
with ``--norm`` normalises them (``layer_norm``), takes two weight matrices of
torch over them and the log probabilities of what follows
(``token_logprobs``), and on the way back

* sums the table's gradient by sorted tokens (the lookup's own gradient,
  ``embedding_grad``), dense and fp32, as the sparsifier takes it;
* sends the largest 1% of it after error feedback (``TopkStep``): here the
  worker applies its own pairs, where many would merge theirs;
* updates the matrices by Muon (``muon_step``), whose Newton-Schulz products
  orthogonalise the momentum.

The data are drawn from a fixed random successor table, one in ten tokens at
random and the last place of every sequence without a successor (a masked
place).  Prints the loss, which falls from log(vocab).

With ``--distill`` a second, smaller model then learns from the first one's
eight largest scores a place instead of the data's successors
(``distillation_loss``); the printed loss is its divergence from them.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_gradient_sparsification_amd as tgs


class Model:
    def __init__(self, vocab, dim, density, seed=0, norm=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sigma):
            return (sigma * torch.randn(*shape, device="cuda", generator=gen)).requires_grad_()

        self.scale = math.sqrt(dim)
        self.table = normal(vocab, dim, sigma=1 / dim)
        self.hidden = normal(dim, dim, sigma=1 / math.sqrt(dim))
        self.output = normal(dim, vocab, sigma=1 / math.sqrt(dim))
        self.matrices = [(w, torch.zeros_like(w)) for w in (self.hidden, self.output)]
        self.gain = torch.ones(dim, device="cuda").requires_grad_() if norm else None
        self.shift = torch.zeros(dim, device="cuda").requires_grad_() if norm else None
        n = self.table.numel()
        self.residual = torch.zeros(n, device="cuda")
        self.topk = tgs.TopkStep(n, max(1, int(density * n)))

    def logits(self, tokens):
        x = tgs.embedding_lookup(tokens, self.table, scale=self.scale)
        if self.gain is not None:
            x = tgs.layer_norm(x, self.gain, self.shift)
        return torch.tanh(x.flatten(0, 1) @ self.hidden) @ self.output

    def alternatives(self, tokens, targets, top):
        """The ``top`` likeliest tokens of every place with a target and their log probabilities; -1 elsewhere."""
        with torch.no_grad():
            r = tgs.token_logprobs(self.logits(tokens), targets.flatten(), top=top)
        return r.top_indices, r.top_logprobs

    def loss(self, tokens, targets, teacher=None):
        """Mean over the places with a target: of -log p(target), or of the divergence from a teacher's alternatives."""
        logits, targets = self.logits(tokens), targets.flatten()
        if teacher is None:
            losses = -tgs.token_logprobs(logits, targets).logprobs
        else:
            losses = tgs.distillation_loss(logits, *teacher)
        return losses.sum() / (targets >= 0).sum()

    def step(self, tokens, targets, lr_table, lr_matrices, teacher=None):
        vectors = [p for p in (self.gain, self.shift) if p is not None]
        for t in (self.table, self.hidden, self.output, *vectors):
            t.grad = None
        loss = self.loss(tokens, targets, teacher)
        loss.backward()
        with torch.no_grad():
            idx, val = self.topk(self.table.grad.view(-1), self.residual)
            self.table.view(-1).index_add_(0, idx, val, alpha=-lr_table)
            for w, momentum in self.matrices:
                # Muon scales a step by sqrt(max(1, out / in)), muon_step by sqrt(max(1, rows / cols)):
                # these matrices are [in, out]
                n_in, n_out = w.shape
                scale = math.sqrt(max(1, n_out / n_in) / max(1, n_in / n_out))
                tgs.muon_step(w, w.grad, momentum, lr=lr_matrices * scale)
            for p in vectors:
                p.sub_(p.grad, alpha=lr_matrices)
        return loss.detach()


def batches(vocab, sequences, length, seed=1):
    """Endless (tokens, targets); -1 marks a place without a target."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    successor = torch.randperm(vocab, device="cuda", generator=gen)
    while True:
        columns = [torch.randint(vocab, (sequences,), device="cuda", generator=gen)]
        for _ in range(length - 1):
            lost = torch.rand(sequences, device="cuda", generator=gen) < 0.1
            drawn = torch.randint(vocab, (sequences,), device="cuda", generator=gen)
            columns.append(torch.where(lost, drawn, successor[columns[-1]]))
        tokens = torch.stack(columns, 1)
        targets = torch.cat([tokens[:, 1:], torch.full_like(tokens[:, :1], -1)], 1)
        yield tokens, targets


def train(steps=60, vocab=4096, dim=256, density=0.01, sequences=64, length=128, report=10, norm=False, teacher=None,
          top=8, model=None):
    model, losses = model or Model(vocab, dim, density, norm=norm), []
    for i, (tokens, targets) in zip(range(steps), batches(vocab, sequences, length)):
        told = teacher.alternatives(tokens, targets, top) if teacher else None
        losses.append(model.step(tokens, targets, lr_table=2.0, lr_matrices=0.02, teacher=told))
        if report and (i % report == 0 or i == steps - 1):
            print("step %3d  loss %.3f" % (i, losses[-1].item()), flush=True)
    model.topk.check()
    return [float(x) for x in losses]


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--vocab", type=int, default=4096)
    p.add_argument("--dim", type=int, default=256)
    p.add_argument("--density", type=float, default=0.01)
    p.add_argument("--norm", action="store_true")
    p.add_argument("--distill", action="store_true")
    a = p.parse_args()
    first = Model(a.vocab, a.dim, a.density, norm=a.norm)
    train(a.steps, a.vocab, a.dim, a.density, model=first)
    if a.distill:
        train(a.steps, a.vocab, a.dim // 2, a.density, norm=a.norm, teacher=first)
