"""A small language model trained end to end against a teacher's top logits
through the sharded step: the token embedding with its gradient (Embedding), the
distillation loss of a head tied to it (HeadDistill), the global gradient norm
and the clipped step (UnitSequence.clip_step), N emulated ranks on one GPU.

Every rank's gradients land in its flat gradient buffers. The table is the
embedding and the head: its view of the buffer first gets the head's gradient,
whole, and then has the embedding's added, in the rows that the batch's tokens
use. The body's parameters (two residual feed-forward blocks and a norm in plain
PyTorch) get theirs through autograd. The teacher is a fixed model of the same
kind, wider, of which only the largest logits of each position are kept.

    python examples/distilled_training.py [--steps 60] [--world 4]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import sharded_fsdp_reduce_gb300 as F  # noqa: E402

VOCAB, DIM, HIDDEN, TOKENS, TOP, TEMPERATURE, IGNORE = 1003, 128, 320, 510, 32, 2.0, -100
SCALE = math.sqrt(DIM)  # of the embedding's rows


def body(p, h):
    """Hidden states [T, DIM] before the head, from the embedding's rows."""
    for k in range(2):
        h = h + torch.relu(h @ p[f"up{k}"]) @ p[f"down{k}"]
    return torch.nn.functional.rms_norm(h, (DIM,), p["norm"])


def make_units(world, device):
    g = torch.Generator().manual_seed(0)
    body_shapes = []
    for k in range(2):
        body_shapes += [(f"up{k}", (DIM, HIDDEN)), (f"down{k}", (HIDDEN, DIM))]
    body_shapes += [("norm", (DIM,))]
    shapes = [[("table", (VOCAB, DIM))], body_shapes]  # the tied table is a unit of its own
    units = []
    for s in shapes:
        u = F.FlatParamUnit(s, world, torch.bfloat16, torch.bfloat16, device=device, n_full=1)
        init = [torch.ones(shape) if n == "norm" else torch.randn(shape, generator=g) * 0.05 for n, shape in s]
        u.load_master([t.to(device) for t in init])
        u.shard_out.copy_(u.master)
        u.all_gather()  # the compute copy before the first forward
        units.append(u)
    return units


class Teacher:
    """A wider table and one hidden layer, fixed."""

    def __init__(self, device, dim=256):
        g = torch.Generator(device=device).manual_seed(7)
        make = lambda *shape: torch.randn(*shape, device=device, generator=g)  # noqa: E731
        self.table, self.mix, self.head = make(VOCAB, dim), make(dim, dim) / math.sqrt(dim), make(VOCAB, dim) * 0.15

    def top(self, tokens):
        """The TOP largest logits of each position and their tokens; padding has none (-1)."""
        logits = torch.tanh(self.table[tokens.clamp(min=0)] @ self.mix) @ self.head.t()
        values, ids = logits.topk(TOP, dim=1)
        ids[tokens == IGNORE] = -1
        return values, ids


def batch(generator, device):
    """Tokens; the last ones are padding."""
    u = torch.rand(TOKENS, device=device, generator=generator)
    tokens = (torch.exp(u * math.log(VOCAB + 1.0)).long() - 1).clamp_(0, VOCAB - 1)  # some are common
    tokens[-10:] = IGNORE
    return tokens


class Student:
    """The model's parts that this package runs, and one rank's pass."""

    def __init__(self, units, device):
        self.units = units
        self.weights = {n: v for u in units for n, v in u.param_views(u.full[0]).items()}
        self.table = F.Embedding(VOCAB, DIM, torch.bfloat16, max_tokens=TOKENS, scale=SCALE, ignore_index=IGNORE,
                                 device=device)
        self.head = F.HeadDistill(VOCAB, DIM, torch.bfloat16, max_tokens=TOKENS, top=TOP, temperature=TEMPERATURE,
                                  device=device)
        self.d_hidden = torch.empty(TOKENS, DIM, dtype=torch.bfloat16, device=device)

    def forward_backward(self, rank, tokens, teacher_logits, teacher_ids, loss=None):
        table, layers = self.units
        d_table = table.param_views(table.grads[rank])["table"]
        layers.grads[rank].zero_()
        grads = layers.param_views(layers.grads[rank])
        leaves = {n: self.weights[n].detach().requires_grad_(True) for n in grads}
        for n, leaf in leaves.items():
            leaf.grad = grads[n]  # autograd adds into the rank's flat buffer
        rows = self.table.forward(tokens, self.weights["table"]).requires_grad_(True)
        hidden = body(leaves, rows)
        loss, _ = self.head.forward_backward(hidden.detach(), self.weights["table"], teacher_logits, teacher_ids,
                                             self.d_hidden, d_table, loss=loss)
        hidden.backward(self.d_hidden)
        self.table.backward(tokens, rows.grad, d_table, accumulate=True)  # after the head's
        return loss


def train(steps=60, world=4, max_norm=1.0, lr=3e-3, device="cuda", report=print):
    units = make_units(world, device)
    model = F.UnitSequence(units)
    student, teacher = Student(units, device), Teacher(device)
    generator = torch.Generator(device=device).manual_seed(1)
    losses = torch.zeros(steps, world, device=device)
    norms = torch.zeros(steps, device=device)
    for t in range(steps):
        for r in range(world):
            tokens = batch(generator, device)
            student.forward_backward(r, tokens, *teacher.top(tokens), loss=losses[t, r])
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
