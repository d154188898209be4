"""One training step around the head, operator by operator: a one-layer language
model with a tied embedding on packed sequences, on one GB300.

    python examples/train_tied_lm.py [--steps 60]

Forward: embedding lookup, a causal attention block over packed sequences, and
the fused linear cross-entropy against the same embedding weight.  Backward: the
head leaves its gradient in an fp32 dW, the attention's gradients go through the
projections, and the embedding's gradient is added to that dW.  Update: the
projections take orthogonalised momentum, the embedding plain momentum.

The data is a noisy cycle over the vocabulary (the next token is usually the
successor), so that the loss has something to fall to.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_cross_entropy_fwd_gb300 as flce  # noqa: E402

IGNORE = -100


class TiedLM:
    """x = E[ids];  y = x + Attn(x Wq, x Wk, x Wv) Wo;  logits = y E^T."""

    def __init__(self, vocab=4096, hidden=512, heads_q=8, heads_kv=2, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads_q, self.heads_kv, self.dim = heads_q, heads_kv, hidden // heads_q

        def init(rows, cols, std):
            return torch.randn(rows, cols, generator=g, device=device) * std

        self.embed = init(vocab, hidden, 0.5 * hidden ** -0.5)
        self.wqkv = init(hidden, (heads_q + 2 * heads_kv) * self.dim, hidden ** -0.5)
        self.wo = init(heads_q * self.dim, hidden, hidden ** -0.5)
        self.scale = hidden ** 0.5 * 0.2
        self.momentum = {n: torch.zeros_like(getattr(self, n)) for n in ("embed", "wqkv", "wo")}

    def loss_and_grads(self, ids, target, cu_seqlens):
        """Mean loss, and the gradients of embed, wqkv and wo in fp32."""
        T, Hq, Hkv, D = ids.shape[0], self.heads_q, self.heads_kv, self.dim
        E, Wqkv, Wo = self.embed.bfloat16(), self.wqkv.bfloat16(), self.wo.bfloat16()
        x = flce.flce_embed_fwd(E, ids, scale=self.scale, ignore_index=IGNORE)
        qkv = (x @ Wqkv).view(T, Hq + 2 * Hkv, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        o, lse = flce.flce_attn_fwd(q, k, v, cu_seqlens)
        flat = o.view(T, Hq * D)
        y = x + flat @ Wo

        loss, _, dy, dE = flce.flce_fwd_bwd_ex(y, E, target, IGNORE)

        dqkv = torch.empty_like(qkv)
        dWo = (flat.T @ dy).float()
        dO = (dy @ Wo.T).view(T, Hq, D)
        flce.flce_attn_bwd(dO, q, k, v, o, lse, cu_seqlens, dq=dqkv[:, :Hq],
                           dk=dqkv[:, Hq:Hq + Hkv], dv=dqkv[:, Hq + Hkv:])
        flat_d = dqkv.view(T, -1)
        dWqkv = (x.T @ flat_d).float()
        dx = dy + flat_d @ Wqkv.T
        # the tied weight's second gradient joins the head's
        flce.flce_embed_bwd(dx, ids, scale=self.scale, ignore_index=IGNORE, dW=dE,
                            accumulate=True)
        return loss, {"embed": dE, "wqkv": dWqkv, "wo": dWo}

    def update(self, grads, lr_embed=5.0, lr_matrix=0.05, beta=0.9):
        for name, grad in grads.items():
            m = self.momentum[name].mul_(beta).add_(grad)
            w = getattr(self, name)
            if name == "embed":
                w.add_(m, alpha=-lr_embed)
            else:
                step = flce.flce_orthogonalize(m)
                w.add_(step.float(), alpha=-lr_matrix * max(1.0, w.shape[0] / w.shape[1]) ** 0.5)


def batch(vocab, lens, seed, device="cuda"):
    """Packed sequences: each token is the one before it plus one (mod vocab), or
    now and then any token; targets are the next tokens, the last of each
    sequence ignored."""
    g = torch.Generator(device=device).manual_seed(seed)
    T = sum(lens)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32,
                      device=device)
    start = torch.randint(0, vocab, (len(lens),), generator=g, device=device)
    pos = torch.arange(T, device=device)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=device),
                                  torch.tensor(lens, device=device))
    ids = (start[seq] + pos - cu[seq].long()) % vocab
    noise = torch.rand(T, generator=g, device=device) < 0.05
    ids = torch.where(noise, torch.randint(0, vocab, (T,), generator=g, device=device), ids)
    target = torch.roll(ids, -1)
    target[cu[1:].long() - 1] = IGNORE
    return ids, target, cu


def train(steps=60, vocab=4096, lens=(700, 333, 1024, 57, 480), log=None):
    """Losses of the steps, each on a new batch."""
    model = TiedLM(vocab=vocab)
    losses = []
    for step in range(steps):
        loss, grads = model.loss_and_grads(*batch(vocab, list(lens), step))
        model.update(grads)
        losses.append(loss)
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:3d}  loss {loss.item():.4f}")
    return [x.item() for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps, log=print)
