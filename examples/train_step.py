"""A small language model trained with the package's operators, one step at a time.

    python examples/train_step.py [steps]

The model looks a token up in an embedding table, passes it through residual
blocks of two matrices each and scores the vocabulary with an output matrix; it
learns a fixed next-token rule on synthetic tokens. A step is what a training
program does around main_grad:

  loss      token_logprobs: log probability of the next token, its entropy, and
            the best alternative (the accuracy is how often that is the token)
  gradient  token_logprobs_backward, in place on the logits
  blocks    plain matrix products; the weight gradients are added to main_grad
  table     accumulate_embedding_wgrad
  update    muon_step for all matrices of the blocks in one call; plain gradient
            descent for the table and the output matrix
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_embedding_weight_amd as ewg  # noqa: E402


class Model:
    """bf16 weights, fp32 main_grad. mats is [2 * blocks, hidden, hidden]."""

    def __init__(self, vocab=1024, hidden=256, blocks=2, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g) * scale).bfloat16().to(device)

        self.table = normal(vocab, hidden, scale=1.0)
        self.mats = normal(2 * blocks, hidden, hidden, scale=hidden ** -0.5)
        self.out = normal(vocab, hidden, scale=hidden ** -0.5)
        self.grads = {n: torch.zeros(getattr(self, n).shape, device=device) for n in ("table", "mats", "out")}
        self.momentum = torch.zeros_like(self.grads["mats"])

    def forward(self, ids):
        """Logits, and what the backward pass needs."""
        h = self.table[ids].float()
        kept = []
        for b in range(0, len(self.mats), 2):
            z = h @ self.mats[b].float().t()
            kept.append((h, z))
            h = h + torch.relu(z) @ self.mats[b + 1].float().t()
        return (h @ self.out.float().t()).bfloat16(), h, kept

    def backward(self, ids, grad_logits, h, kept):
        """Adds every weight's gradient to its main_grad."""
        d = grad_logits.float()
        self.grads["out"] += d.t() @ h
        dh = d @ self.out.float()
        for b, (x, z) in reversed(list(enumerate(kept))):
            self.grads["mats"][2 * b + 1] += dh.t() @ torch.relu(z)
            dz = (dh @ self.mats[2 * b + 1].float()) * (z > 0)
            self.grads["mats"][2 * b] += dz.t() @ x
            dh = dh + dz @ self.mats[2 * b].float()
        ewg.accumulate_embedding_wgrad(ids, dh, self.grads["table"])

    def update(self, lr):
        ewg.muon_step(self.mats, self.grads["mats"], self.momentum, lr=lr, weight_decay=0.01)
        for n in ("table", "out"):
            getattr(self, n).add_(self.grads[n].bfloat16(), alpha=-50 * lr)
        for t in self.grads.values():
            t.zero_()


def batch(tokens, vocab, step, device="cuda"):
    """Tokens and the ones that follow them; one position in sixteen has none."""
    g = torch.Generator().manual_seed(1000 + step)
    ids = torch.randint(0, vocab, (tokens,), generator=g)
    following = (ids * 37 + 11) % vocab
    following[::16] = -100
    return ids.to(device), following.to(device)


def loss_and_gradient(model, ids, following, entropy_weight=0.01):
    """Mean loss, share of tokens whose best alternative is the next token; main_grad
    holds the gradients afterwards."""
    logits, h, kept = model.forward(ids)
    r = ewg.token_logprobs(logits, following, top_k=1)
    asked = following >= 0
    n = asked.sum()
    weight = asked.float() / n
    loss = -(weight * (r.logprobs + entropy_weight * r.entropy)).sum()
    right = (r.top_ids[:, 0] == following).sum() / n
    ewg.token_logprobs_backward(logits, following, r.logsumexp, r.entropy, -weight, -entropy_weight * weight, out=logits)
    model.backward(ids, logits, h, kept)
    return loss, right


def train(steps=40, tokens=4096, lr=0.02, model=None):
    model = model or Model()
    vocab = model.table.shape[0]
    history = []
    for step in range(steps):
        ids, following = batch(tokens, vocab, step)
        loss, right = loss_and_gradient(model, ids, following)
        model.update(lr)
        history.append((float(loss), float(right)))
    return history


if __name__ == "__main__":
    for step, (loss, right) in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)):
        print(f"step {step:3d}  loss {loss:7.4f}  right {100 * right:5.1f} %", flush=True)
