"""The token embedding, the distillation loss, the global norm and the clipped
step as one training loop (examples/distilled_training.py): that it runs, and
one rank's gradients against their definition."""
import os
import sys

import pytest
import torch

from test_distill_gpu import check as check_distilled, reference as distilled
from test_embedding_gpu import check_lookup, gradient

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def example():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import distilled_training
    return distilled_training


def test_it_runs(example):
    losses, norms = example.train(steps=5, world=2, report=lambda s: None)
    assert bool(torch.isfinite(losses).all()) and bool((losses > 0).all()) and bool((norms > 0).all())


def test_gradients_against_the_definition(example):
    """One rank's pass: the body is torch's on both sides, in bf16, so its inputs
    and gradients are the same bits; the embedding's rows, the loss and the tied
    table's gradient are held to fp64 with the bounds of their own tests (a
    table's gradient is rounded twice: the head's, then with the embedding's)."""
    units = example.make_units(2, DEV)
    student, teacher = example.Student(units, DEV), example.Teacher(DEV)
    tokens = example.batch(torch.Generator(device=DEV).manual_seed(5), DEV)
    values, ids = teacher.top(tokens)
    loss = student.forward_backward(1, tokens, values, ids).detach()
    table, layers = units
    got = {**table.param_views(table.grads[1]), **layers.param_views(layers.grads[1])}
    w = student.weights["table"]

    rows = student.table.forward(tokens, w)
    check_lookup(rows, tokens, w, "bf16", example.SCALE)
    rows.requires_grad_(True)
    leaves = {n: student.weights[n].detach().requires_grad_(True) for n in layers.names}
    hidden = example.body(leaves, rows)
    ref = distilled(hidden.detach(), w, values, ids, example.TEMPERATURE)
    check_distilled(ref, "bf16", (example.VOCAB, example.TOKENS), loss, ref["tok"].float(), student.d_hidden)
    assert torch.equal(ref["valid"], tokens != example.IGNORE)
    hidden.backward(student.d_hidden)
    for n, leaf in leaves.items():
        assert torch.equal(got[n], leaf.grad), n
    total, size, count = gradient(tokens, rows.grad, example.VOCAB, example.SCALE)
    want = ref["dw"] + total
    u = 2.0 ** -8
    bound = 1.1 * ((u + 2.0 ** -11) * ref["sw"] + ref["ew"]) + u * ref["dw"].abs()  # the head's
    bound += 1.01 * 2.0 ** -24 * (count + 3)[:, None] * size + u * want.abs() + 1e-37
    bound *= 1 + 2 * u  # (the second rounding is of what the first one left)
    err = (got["table"].double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    # both ends' gradients are in the table: without either it is far off
    for part in (ref["dw"], total):
        assert float((got["table"].double() - part).norm()) > 10 * float(bound.norm())


def test_a_captured_pass(example):
    """The package's parts of a pass in one graph: lookup, loss with gradients,
    the embedding's gradient on top; replayed on other data, the bits of the
    eager calls."""
    units = example.make_units(1, DEV)
    student, teacher = example.Student(units, DEV), example.Teacher(DEV)
    w = student.weights["table"]
    tokens = example.batch(torch.Generator(device=DEV).manual_seed(1), DEV)
    values, ids = teacher.top(tokens)
    rows = torch.empty(example.TOKENS, example.DIM, dtype=torch.bfloat16, device=DEV)
    d_table = torch.empty_like(w)

    def one_pass():
        student.table.forward(tokens, w, out=rows)
        student.head.forward_backward(rows, w, values, ids, student.d_hidden, d_table, loss=one_pass.loss,
                                      token_loss=one_pass.token_loss)
        student.table.backward(tokens, student.d_hidden, d_table, accumulate=True)

    one_pass.loss = torch.empty((), device=DEV)
    one_pass.token_loss = torch.empty(example.TOKENS, device=DEV)
    one_pass()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_pass()
    for seed in (2, 3):
        tokens.copy_(example.batch(torch.Generator(device=DEV).manual_seed(seed), DEV))
        new = teacher.top(tokens)
        values.copy_(new[0]), ids.copy_(new[1])
        one_pass()
        want = [t.clone() for t in (rows, one_pass.loss, student.d_hidden, d_table)]
        for t in (rows, one_pass.loss, student.d_hidden, d_table):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (rows, one_pass.loss, student.d_hidden, d_table)))
