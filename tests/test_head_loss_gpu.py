"""The head loss (fsdp_head_loss, HeadLoss) against its definition in fp64.

Tolerances, derived from the operations (u = 2^-8 bf16, 2^-11 fp16 unit
roundoff; A = max_v sum_k |x_k w_k| of a row):
* logits: fp32 products and sums, 8 sqrt(D) 2^-23 A; the exponential and the
  sums behind lse 2^-20 max(1, |lse|). A token's loss has both.
* a gradient element: its sum of |d||w| (or |d||x|) times d's error: one
  rounding to the head's type (u), one to fp16 before it (2^-11), the logit's
  error; 10 % for second-order terms; and the output's own rounding.
* fp32 heads: the logit's error, 2^-20 for the exponential, the split
  products and sums 4 sqrt(K) 2^-23, the output 2^-23.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
IGNORE = -100


@pytest.fixture(scope="module")
def F():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sharded_fsdp_reduce_gb300 as F
    return F


def inputs(T, V, D, dt, seed=0, std=0.05, ignored="tail"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(T, D, device=DEV).normal_(generator=g).to(DT[dt])
    w = (torch.empty(V, D, device=DEV).normal_(generator=g) * std).to(DT[dt])
    y = torch.randint(0, V, (T,), device=DEV, generator=g)
    if ignored == "tail":
        y[T - T // 4:] = IGNORE
    elif ignored == "some":
        y[torch.rand(T, device=DEV, generator=g) < 0.3] = IGNORE
    elif ignored == "all":
        y[:] = IGNORE
    return x, w, y


def reference(x, w, y, reduction="mean", grad_scale=1.0):
    """Loss, token losses, lse, gradients, and the sums that bound their errors, in fp64."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    valid = y != IGNORE
    at = torch.where(valid, y, 0)
    tok = torch.where(valid, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    n = max(int(valid.sum()), 1) if reduction == "mean" else 1
    d = torch.exp(z - lse[:, None])
    d.scatter_add_(1, at[:, None], torch.full((len(y), 1), -1.0, dtype=torch.float64, device=DEV))
    d *= valid[:, None]
    g = grad_scale / n
    a = (x.abs() @ w.abs().t()).amax(1) if len(y) else x.new_zeros(0)
    return dict(loss=tok.sum() / n, tok=tok, lse=lse, dx=g * (d @ w), dw=g * (d.t() @ x), n=n, a=a,
                sx=abs(g) * (d.abs() @ w.abs()), sw=abs(g) * (d.abs().t() @ x.abs()), valid=valid)


def check(ref, dt, D, K, loss, tok, dx=None, dw=None):
    logit = 8 * math.sqrt(D) * 2.0 ** -23 * ref["a"]
    tol = logit + 2.0 ** -20 * ref["lse"].abs().clamp(min=1)
    err = (tok.double() - ref["tok"]).abs()
    assert bool((err <= tol).all()), f"token loss off by {err.max():.3g}, allowed {tol[err.argmax()]:.3g}"
    assert bool((tok[~ref["valid"]] == 0).all())
    worst = float(tol.max()) if len(tol) else 0.0
    scale = len(tol) / ref["n"]
    assert abs(float(loss) - float(ref["loss"])) <= worst * max(1.0, scale) + 2.0 ** -23 * abs(float(ref["loss"]))
    le = float(logit.max()) if len(tol) else 0.0
    for got, want, size, k in ((dx, ref["dx"], ref["sx"], K[0]), (dw, ref["dw"], ref["sw"], K[1])):
        if got is None:
            continue
        if dt == "f32":
            rel = le + 2.0 ** -20 + 4 * math.sqrt(k) * 2.0 ** -23
            bound = rel * size + 2.0 ** -23 * want.abs() + 1e-37
        else:
            bound = 1.1 * (U[dt] + 2.0 ** -11 + le) * size + U[dt] * want.abs()
            bound += 2.0 ** -25 if dt == "f16" else 1e-37  # half the smallest subnormal step
        err = (got.double() - want).abs()
        over = err > bound
        assert not bool(over.any()), (f"{int(over.sum())} of {over.numel()} gradient elements beyond the bound, "
                                      f"first at {over.nonzero()[0].tolist()}, worst ratio {float((err / bound).max()):.3g}")


def run(F, x, w, y, grad=True, **kw):
    T, V = len(y), w.shape[0]
    head = F.HeadLoss(V, w.shape[1], x.dtype, T, grad=grad, reduction=kw.pop("reduction", "mean"),
                      band=kw.pop("band", 0))
    waits = torch.zeros(1, dtype=torch.int32, device=DEV)
    if not grad:
        loss, tok = head.forward(x, w, y, wait_timeouts=waits)
        dx = dw = None
    else:
        dx = kw.pop("dx", None)
        dw = kw.pop("dw", None)
        dx = torch.full_like(x, float("nan")) if dx is None else dx
        dw = torch.full_like(w, float("nan")) if dw is None else dw
        loss, tok = head.forward_backward(x, w, y, dx, dw, wait_timeouts=waits, **kw)
    torch.cuda.synchronize()
    assert int(waits.item()) == 0
    return loss, tok, dx, dw


SIZES = [  # tokens, vocab, dim: tiles' edges on both sides, odd ones, one of everything
    (1, 1, 8), (1, 1000, 64), (2, 257, 72), (31, 128, 128), (33, 129, 8), (128, 256, 64), (129, 1003, 200),
    (255, 511, 264), (257, 640, 512), (300, 5000, 768), (1021, 3001, 320),
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_losses(F, T, V, D, dt):
    x, w, y = inputs(T, V, D, dt)
    loss, tok, _, _ = run(F, x, w, y, grad=False)
    check(reference(x, w, y), dt, D, (V, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_gradients(F, T, V, D, dt):
    x, w, y = inputs(T, V, D, dt, ignored="some")
    loss, tok, dx, dw = run(F, x, w, y)
    check(reference(x, w, y), dt, D, (V, T), loss, tok, dx, dw)
