"""The head loss, the global norm and the clipped step as one training loop
(examples/clipped_training.py), and one of its steps against plain autograd."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def example():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import clipped_training
    return clipped_training


def test_the_loss_falls(example):
    losses, norms = example.train(steps=40, world=2, report=lambda s: None)
    assert bool(torch.isfinite(losses).all()) and bool((norms > 0).all())
    # log(1003) = 6.91 before training; the rule can be learnt
    assert 6.5 < float(losses[0]) < 7.5
    assert float(losses[-5:].mean()) < 0.75 * float(losses[0])


def test_one_step_against_autograd(example):
    """The same step with torch's own loss, norm and clipping in fp32 on one replica."""
    F = example.F
    world, max_norm, lr = 2, 0.5, 1e-2
    units = example.make_units(world, DEV)
    weights = {**units[0].param_views(units[0].full[0]), **units[1].param_views(units[1].full[0])}
    ref = {n: w.detach().float().requires_grad_(True) for n, w in weights.items()}
    masters = {n: v.clone() for u in units for n, v in u.param_views(u.master).items()}
    head = F.HeadLoss(example.VOCAB, example.DIM, torch.bfloat16, example.TOKENS, ignore_index=example.IGNORE)
    generator = torch.Generator(device=DEV).manual_seed(5)
    d_hidden = torch.empty(example.TOKENS, example.DIM, dtype=torch.bfloat16, device=DEV)
    total = 0.0
    for r in range(world):
        tokens, targets = example.batch(generator, DEV)
        units[0].grads[r].zero_()
        grads = units[0].param_views(units[0].grads[r])
        leaves = {n: weights[n].detach().requires_grad_(True) for n in grads}
        for n, leaf in leaves.items():
            leaf.grad = grads[n]
        hidden = example.body(leaves, tokens)
        loss, _ = head.forward_backward(hidden.detach(), weights["head"], targets, d_hidden,
                                        units[1].param_views(units[1].grads[r])["head"])
        hidden.backward(d_hidden)
        want = torch.nn.functional.cross_entropy(example.body(ref, tokens) @ ref["head"].t(), targets,
                                                 ignore_index=example.IGNORE)
        # the body runs in bf16 here and in fp32 there: 2^-8 per operation
        assert abs(float(loss) - float(want)) < 0.02
        total = total + want / world
    total.backward()
    want_norm = float(torch.linalg.vector_norm(torch.stack([p.grad.norm() for p in ref.values()])))
    norm = F.UnitSequence(units).clip_step(F.AdamWHParams(lr, step=1), max_norm)
    torch.cuda.synchronize()
    assert want_norm > max_norm  # the step is clipped
    assert abs(float(norm) - want_norm) < 0.03 * want_norm
    # the first AdamW step moves every weight by lr along its gradient's sign
    # (eps aside): where the gradient is well above bf16's noise they agree
    for n, p in ref.items():
        view = next(u.param_views(u.master)[n] for u in units if n in u.names)
        moved = (view - masters[n]).sign()
        sure = p.grad.abs() > 0.1 * p.grad.abs().max()
        assert int(sure.sum()) > 0 and bool((moved[sure] == -p.grad.sign()[sure]).float().mean() > 0.99), n
