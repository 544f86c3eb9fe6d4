"""A small language model trained end to end through the sharded step: the
head's loss and gradients (HeadLoss), the global gradient norm and the clipped
step (UnitSequence.clip_step), N emulated ranks on one GPU.

Every rank's gradients land in its flat gradient buffers: the body's through
autograd (the parameters' .grad are views of them), the head's straight from
the loss. The body is an embedding, two residual feed-forward blocks and a
norm in plain PyTorch; the data is a noisy successor rule over the vocabulary.

    python examples/clipped_training.py [--steps 60] [--world 4]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import sharded_fsdp_reduce_gb300 as F  # noqa: E402

VOCAB, DIM, HIDDEN, TOKENS, IGNORE = 1003, 128, 320, 510, -100


def body(p, tokens):
    """Hidden states [T, DIM] before the head."""
    h = p["embed"][tokens]
    for k in range(2):
        h = h + torch.relu(h @ p[f"up{k}"]) @ p[f"down{k}"]
    return torch.nn.functional.rms_norm(h, (DIM,), p["norm"])


def make_units(world, device):
    g = torch.Generator().manual_seed(0)
    body_shapes = [("embed", (VOCAB, DIM))]
    for k in range(2):
        body_shapes += [(f"up{k}", (DIM, HIDDEN)), (f"down{k}", (HIDDEN, DIM))]
    body_shapes += [("norm", (DIM,))]
    shapes = [body_shapes, [("head", (VOCAB, DIM))]]  # the head is a unit of its own
    units = []
    for s in shapes:
        u = F.FlatParamUnit(s, world, torch.bfloat16, torch.bfloat16, device=device, n_full=1)
        init = [torch.ones(shape) if n == "norm" else torch.randn(shape, generator=g) * 0.05 for n, shape in s]
        u.load_master([t.to(device) for t in init])
        u.shard_out.copy_(u.master)
        u.all_gather()  # the compute copy before the first forward
        units.append(u)
    return units


def batch(generator, device):
    """Tokens and their successors; the last ones are padding."""
    tokens = torch.randint(0, VOCAB, (TOKENS,), device=device, generator=generator)
    targets = (7 * tokens + 3) % VOCAB
    noise = torch.rand(TOKENS, device=device, generator=generator) < 0.05
    targets[noise] = tokens[noise]
    targets[-10:] = IGNORE
    return tokens, targets


def train(steps=60, world=4, max_norm=1.0, lr=3e-3, device="cuda", report=print):
    units = make_units(world, device)
    model = F.UnitSequence(units)
    weights = {**units[0].param_views(units[0].full[0]), **units[1].param_views(units[1].full[0])}
    head = F.HeadLoss(VOCAB, DIM, torch.bfloat16, max_tokens=TOKENS, ignore_index=IGNORE, device=device)
    d_hidden = torch.empty(TOKENS, DIM, dtype=torch.bfloat16, device=device)
    generator = torch.Generator(device=device).manual_seed(1)
    losses = torch.zeros(steps, world, device=device)
    norms = torch.zeros(steps, device=device)
    for t in range(steps):
        for r in range(world):
            tokens, targets = batch(generator, device)
            units[0].grads[r].zero_()
            grads = units[0].param_views(units[0].grads[r])
            leaves = {n: weights[n].detach().requires_grad_(True) for n in grads}
            for n, leaf in leaves.items():
                leaf.grad = grads[n]  # autograd adds into the rank's flat buffer
            hidden = body(leaves, tokens)
            head.forward_backward(hidden.detach(), weights["head"], targets, d_hidden,
                                  units[1].param_views(units[1].grads[r])["head"], loss=losses[t, r])
            hidden.backward(d_hidden)
        model.clip_step(F.AdamWHParams(lr, beta2=0.95, weight_decay=0.01, step=t + 1), max_norm, norm=norms[t])
    for t in range(0, steps, max(1, steps // 10)):
        report(f"step {t:4d}  loss {float(losses[t].mean()):.4f}  gradient norm {float(norms[t]):.4f}")
    report(f"last       loss {float(losses[-1].mean()):.4f}  gradient norm {float(norms[-1]):.4f}")
    return losses.mean(1), norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--world", type=int, default=4)
    ap.add_argument("--max-norm", type=float, default=1.0)
    a = ap.parse_args()
    train(a.steps, a.world, a.max_norm)
