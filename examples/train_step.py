"""A training step whose every result is reproducible, bit for bit.

A one-block language model on synthetic data -- tied token embedding, attention with normed
and rotated queries and keys, cross entropy over the vocabulary -- trained for a few steps
with the library's operators end to end:

    embed_forward -> qk_norm_rope_forward -> attn_forward -> linear_xent_forward
    linear_xent_backward -> attn_backward (a DASH order) -> qk_norm_rope_backward ->
    embed_backward (into the tied table's gradient) -> grad_clip

Only the three projections are torch matrix products. Every run from one seed gives the same
parameters to the last bit:

    python examples/train_step.py --steps 20 --runs 2
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import reproducible_deterministic_attn_gb300 as da  # noqa: E402


class Model:
    """fp32 parameters with bf16 copies that the step computes with."""

    def __init__(self, vocab: int, width: int, heads: int, seed: int, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std

        self.vocab, self.heads, self.head_dim = vocab, heads, width // heads
        self.scale = math.sqrt(width)                # of the embedding
        self.master = {
            "embed": randn(vocab, width, std=width ** -0.5),
            "qkv": randn(3 * width, width, std=width ** -0.5),
            "out": randn(width, width, std=width ** -0.5),
            "wq": torch.ones(self.head_dim, device=device),
            "wk": torch.ones(self.head_dim, device=device),
        }
        self.refresh()

    def refresh(self):
        self.p = {n: t if t.dim() == 1 else t.bfloat16() for n, t in self.master.items()}


class Trainer:
    """The step's workspaces and plan are made once, as its sizes do not change."""

    def __init__(self, model: Model, batch: int, seqlen: int, lr: float = 1.0, max_norm: float = 1.0):
        m, self.model, self.lr, self.max_norm = model, model, lr, max_norm
        B, S, H, D = batch, seqlen, m.heads, m.head_dim
        dev = m.master["embed"].device
        self.shape = (B, S, H, D)
        self.cos, self.sin = da.rope_table(S, D, device=dev)
        self.grads = {n: torch.empty_like(t) for n, t in m.master.items()}
        self.plan = da.grad_clip_plan(self.grads.values())
        self.ws = {
            "attn": da.new_workspace(B, S, H, D, dev),
            "xent": da.new_linear_xent_workspace(B * S, m.vocab, H * D, dev),
            "qk": da.new_qk_norm_rope_workspace(B, S, H, H, D, dev),
            "embed": da.new_embed_workspace(B * S, m.vocab, H * D, dev),
        }

    def step(self, ids, targets):
        """One optimizer step on int ids, targets [B, S]; returns the mean loss and the norm."""
        m, p, g, ws = self.model, self.model.p, self.grads, self.ws
        B, S, H, D = self.shape
        T, W = B * S, H * D
        qk = (p["wq"], p["wk"], self.cos, self.sin)
        att_scale = 1.0 / math.sqrt(D)

        x = da.embed_forward(p["embed"], ids, m.scale).view(T, W)
        qkv = (x @ p["qkv"].t()).view(B, S, 3 * H, D)
        q0, k0, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:].contiguous()
        q, k = da.qk_norm_rope_forward(q0, k0, *qk)
        o, lse = da.attn_forward(q, k, v, att_scale, causal=True)
        h = x + o.view(T, W) @ p["out"].t()
        y = targets.reshape(T)
        loss, zlse = da.linear_xent_forward(h, p["embed"], y, workspace=ws["xent"], check=False)

        counted = y != -100
        dloss = counted.float() / counted.sum()
        dh, _ = da.linear_xent_backward(h, p["embed"], y, zlse, dloss, dw=g["embed"], workspace=ws["xent"],
                                        check=False)
        g["out"].copy_(dh.t() @ o.view(T, W))
        do = (dh @ p["out"]).view(B, S, H, D)
        order = "symmetric_shift" if S % 256 == 0 else "descending"
        dq, dk, dv = da.attn_backward(q, k, v, o, do, lse, att_scale, True, order, 1, ws["attn"], check=False)
        dqkv = torch.empty_like(qkv)
        _, _, dwq, dwk = da.qk_norm_rope_backward(dq, dk, q0, k0, *qk, dq=dqkv[:, :, :H], dk=dqkv[:, :, H:2 * H],
                                                  workspace=ws["qk"], check=False)
        dqkv[:, :, 2 * H:] = dv
        dqkv = dqkv.view(T, 3 * W)
        g["qkv"].copy_(dqkv.t() @ x)
        g["wq"].copy_(dwq)
        g["wk"].copy_(dwk)
        dx = dh + dqkv @ p["qkv"]
        # the table is tied: its other gradient is added to what the loss left
        da.embed_backward(dx.view(B, S, W), ids, m.vocab, m.scale, dtable=g["embed"], accumulate=True,
                          workspace=ws["embed"], check=False)

        norm, _ = da.grad_clip(self.plan, self.max_norm)
        for n, t in m.master.items():
            t.add_(g[n], alpha=-self.lr)
        m.refresh()
        return (loss * dloss).sum(), norm

    def check(self):
        """Raises what any step since the last check reported from the device."""
        for name, w in self.ws.items():
            status = da.dash_attn_get_status(w)
            if status != da.DASH_OK:
                raise da.DashError(status, name)


def train(steps: int, batch: int = 2, seqlen: int = 256, vocab: int = 1000, width: int = 256, heads: int = 4,
          seed: int = 0):
    """Trains from the seed; returns (losses, parameters)."""
    model = Model(vocab, width, heads, seed)
    trainer = Trainer(model, batch, seqlen)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    follows = torch.randperm(vocab, generator=g, device="cuda")       # what there is to learn
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, vocab, (batch, seqlen), generator=g, device="cuda")
        targets = follows[ids]
        targets[:, -1] = -100
        loss, _ = trainer.step(ids, targets)
        losses.append(loss)
    trainer.check()
    return [float(x) for x in losses], model.master


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--runs", type=int, default=2)
    a = ap.parse_args()
    first = None
    for run in range(a.runs):
        losses, params = train(a.steps)
        print(f"run {run}: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
        if first is None:
            first = (losses, params)
        else:
            same = losses == first[0] and all(torch.equal(params[n], first[1][n]) for n in params)
            print("  equal to the first run in every bit" if same else "  DIFFERS from the first run")
            if not same:
                raise SystemExit(1)


if __name__ == "__main__":
    main()
