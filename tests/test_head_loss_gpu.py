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


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 17, 24, 25])
@pytest.mark.parametrize("V,D", [(5003, 768), (129, 100), (33, 3)])
def test_losses_of_a_few_rows(F, T, V, D, dt):
    x, w, y = inputs(T, V, D, dt, seed=T, ignored="some" if T > 4 else None)
    loss, tok, _, _ = run(F, x, w, y, grad=False)
    check(reference(x, w, y), dt, D, (V, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", [(5, 300, 65), (200, 1001, 129), (130, 515, 1)])
def test_dims_that_tma_cannot_address(F, T, V, D, dt):
    x, w, y = inputs(T, V, D, dt, seed=5, std=0.2)
    loss, tok, dx, dw = run(F, x, w, y)
    check(reference(x, w, y), dt, D, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off,pad", [(0, 8), (8, 24), (1, 0), (3, 5), (4, 4), (2, 6)])
def test_views_at_any_offset_and_stride(F, off, pad, dt):
    T, V, D = 140, 700, 136
    x0, w0, y = inputs(T, V, D, dt, seed=6)

    def place(rows, src=None):
        buf = torch.full((off + rows * (D + pad) + 64,), 7.0, dtype=DT[dt], device=DEV)
        v = buf[off:off + rows * (D + pad)].view(rows, D + pad)[:, :D]
        if src is not None:
            v.copy_(src)
        return buf, v

    _, x = place(T, x0)
    _, w = place(V, w0)
    bx, dx = place(T)
    bw, dw = place(V)
    assert pad == 0 or not dx.is_contiguous()
    ref = reference(x0, w0, y)
    loss, tok, _, _ = run(F, x, w, y, dx=dx, dw=dw)
    check(ref, dt, D, (V, T), loss, tok, dx, dw)
    for buf, v, rows in ((bx, dx, T), (bw, dw, V)):  # nothing beside the gradients is written
        v.zero_()
        assert int((buf != 0).sum()) == buf.numel() - rows * D
    loss, tok, _, _ = run(F, x, w, y, grad=False)
    check(ref, dt, D, (V, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,band", [(700, 256), (513, 512), (300, 100), (257, 1)])
def test_bands_of_tokens(F, T, band, dt):
    if band == 1 and dt != "bf16":
        T = 9
    V, D = 777, 200
    x, w, y = inputs(T, V, D, dt, seed=7, ignored="some")
    loss, tok, dx, dw = run(F, x, w, y, band=band)
    check(reference(x, w, y), dt, D, (V, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, x, w, y, grad=False, band=band)
    check(reference(x, w, y), dt, D, (V, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_band_smaller_than_a_few_rows(F, dt):
    for T, band in ((3, 1), (4, 2), (20, 7)):
        x, w, y = inputs(T, 300, 64, dt, seed=T)
        loss, tok, _, _ = run(F, x, w, y, grad=False, band=band)
        check(reference(x, w, y), dt, 64, (300, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_split_products(F, dt):
    # few tiles of a long K: the hidden gradient over the vocabulary, the
    # weight gradient over the tokens
    for T, V, D in ((100, 9000, 64), (3000, 200, 64)):
        x, w, y = inputs(T, V, D, dt, seed=8)
        loss, tok, dx, dw = run(F, x, w, y)
        check(reference(x, w, y), dt, D, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("dt,scale", [("bf16", 1.0), ("f16", 1024.0), ("f32", 0.125)])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_reduction_and_loss_scale(F, dt, scale, reduction):
    T, V, D = 90, 1500, 96
    if dt == "f16" and reduction == "sum":
        scale = 4.0  # the gradients have to fit fp16
    x, w, y = inputs(T, V, D, dt, seed=9, ignored="some")
    loss, tok, dx, dw = run(F, x, w, y, reduction=reduction, grad_scale=scale)
    check(reference(x, w, y, reduction, scale), dt, D, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 200])
def test_no_row_counts(F, T, dt):
    x, w, y = inputs(T, 600, 64, dt, ignored="all")
    loss, tok, dx, dw = run(F, x, w, y)
    assert float(loss) == 0.0 and not bool(tok.any()) and not bool(dx.any()) and not bool(dw.any())
    assert float(run(F, x, w, y, grad=False)[0]) == 0.0


def test_no_tokens(F):
    x, w, y = inputs(0, 100, 64, "bf16", ignored=None)
    loss, tok, dx, dw = run(F, x, w, y)
    assert float(loss) == 0.0 and tok.numel() == 0 and not bool(dw.any())


def test_either_gradient_alone(F):
    x, w, y = inputs(150, 900, 128, "bf16")
    head = F.HeadLoss(900, 128, torch.bfloat16, 150)
    both = [torch.empty_like(x), torch.empty_like(w)]
    head.forward_backward(x, w, y, *both)
    one = torch.empty_like(x)
    head.forward_backward(x, w, y, one, None)
    assert torch.equal(one, both[0])
    two = torch.empty_like(w)
    head.forward_backward(x, w, y, None, two)
    assert torch.equal(two, both[1])


@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_targets_outside_the_vocabulary_show_as_nan(F, T, dt):
    V, D = 500, 64
    for bad in (V, -1, 2 ** 40):
        x, w, y = inputs(T, V, D, dt, ignored=None)
        good = run(F, x, w, y)[1]
        y[2] = bad
        loss, tok, dx, dw = run(F, x, w, y)
        assert math.isnan(float(loss)) and math.isnan(float(tok[2])) and bool(torch.isnan(dx[2]).all())
        keep = torch.arange(T, device=DEV) != 2
        assert torch.equal(tok[keep], good[keep])
        assert not bool(torch.isnan(dx[keep]).any()) and bool(torch.isnan(dw).all())
        assert math.isnan(float(run(F, x, w, y, grad=False)[0]))


@pytest.mark.parametrize("T", [4, 150])
def test_nan_in_a_row_stays_in_its_row(F, T):
    x, w, y = inputs(T, 400, 64, "bf16", ignored=None)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y[2] = IGNORE  # not finite, and ignored: neither its loss nor a gradient of its own
    loss, tok, dx, dw = run(F, x, w, y)
    assert math.isnan(float(loss)) and math.isnan(float(tok[1])) and float(tok[2]) == 0.0
    assert bool(torch.isnan(dx[1]).all()) and not bool(dx[2].any())
    rest = torch.arange(T, device=DEV) > 2
    assert not bool(torch.isnan(tok[rest]).any()) and not bool(torch.isnan(dx[rest]).any())
    assert math.isnan(float(run(F, x, w, y, grad=False)[0]))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [4, 8, 24, 25, 300])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_counted_row_that_is_not_finite(F, T, bad, dt):
    """An infinite hidden value makes some logit +inf or NaN, or all -inf: its
    row has no loss in any type and at any number of rows, nor has the sum."""
    V, D = 500, 64
    x, w, y = inputs(T, V, D, dt, ignored=None)
    good = run(F, x, w, y, grad=False)[1]
    x[3, 5] = bad
    keep = torch.arange(T, device=DEV) != 3
    loss, tok, _, _ = run(F, x, w, y, grad=False)
    assert math.isnan(float(loss)) and math.isnan(float(tok[3]))
    assert torch.equal(tok[keep], good[keep])
    loss, tok, dx, dw = run(F, x, w, y)
    assert math.isnan(float(loss)) and math.isnan(float(tok[3]))
    assert bool(torch.isnan(dx[3]).all()) and bool(torch.isnan(dw).all())
    assert not bool(torch.isnan(dx[keep]).any()) and not bool(torch.isnan(tok[keep]).any())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [4, 8, 24, 25, 300])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_a_weight_that_is_infinite(F, T, bad, dt):
    """Rows whose logit it makes +inf have no loss; for the others, at -inf,
    its column is as if it were not there. With infinities of both signs in a
    logit's products, nothing has a loss."""
    V, D = 500, 64
    x, w, y = inputs(T, V, D, dt, ignored=None)
    y[y == 77] = 78
    w[77, 9] = bad
    x[0, 9], x[1, 9] = 0.5, -0.5  # (few rows might all have one sign)
    up = x[:, 9] * bad > 0
    assert bool(up.any()) and bool((~up).any())
    cols = torch.arange(V, device=DEV) != 77
    ref = reference(x[~up], w[cols], torch.where(y > 77, y - 1, y)[~up])
    logit = 8 * math.sqrt(D) * 2.0 ** -23 * ref["a"] + 2.0 ** -20 * ref["lse"].abs().clamp(min=1)
    for grad in (False, True):
        tok = run(F, x, w, y, grad=grad)[1]
        assert bool(torch.isnan(tok[up]).all())
        assert bool(((tok[~up].double() - ref["tok"]).abs() <= logit).all())
    w[300:310] = bad
    assert bool(torch.isnan(run(F, x, w, y, grad=False)[1]).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,band", [(3, 0), (64, 0), (65, 0), (300, 0), (600, 256)])
def test_what_lies_in_ignored_rows_does_not_matter(F, T, band, dt):
    V, D = 700, 136
    x, w, y = inputs(T, V, D, dt, ignored="some", seed=3)
    y[0], y[1] = 5, IGNORE
    ref = reference(x, w, y)
    dirty = x.clone()
    junk = torch.tensor([float("nan"), float("inf"), -float("inf"), 6e4], device=DEV).to(DT[dt])
    dirty[y == IGNORE] = junk.repeat(D // 4)
    loss, tok, dx, dw = run(F, dirty, w, y, band=band)
    check(ref, dt, D, (V, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, dirty, w, y, grad=False, band=band)
    check(ref, dt, D, (V, T), loss, tok)


@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (7, 65, 127), (16, 640, 256), (33, 1001, 131), (64, 3000, 516), (65, 200, 64)])
def test_gradients_of_a_few_fp32_rows(F, T, V, D):
    x, w, y = inputs(T, V, D, "f32", seed=T, ignored="some" if T > 4 else None, std=0.2)
    loss, tok, dx, dw = run(F, x, w, y)
    ref = reference(x, w, y)
    check(ref, "f32", D, (V, T), loss, tok, dx, dw)
    a = run(F, x, w, y)
    assert torch.equal(a[2], dx) and torch.equal(a[3], dw)
    loss, tok, dx, dw = run(F, x, w, y, reduction="sum", grad_scale=3.0)
    check(reference(x, w, y, "sum", 3.0), "f32", D, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("T", [2, 130])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_vocabulary_entries_that_cannot_be_drawn(F, T, dt):
    # columns whose logits are minus infinity (a masked part of the
    # vocabulary), whole tiles of them among them
    V, D = 900, 64
    x, w, y = inputs(T, V, D, dt, ignored=None)
    x = x.abs() + 0.1
    y %= 100
    w[300:850] = -float("inf")
    keep = torch.cat([torch.arange(300), torch.arange(850, V)]).to(DEV)
    ref = reference(x, w[keep], y)
    loss, tok, _, _ = run(F, x, w, y, grad=False)
    check(ref, dt, D, (V, T), loss, tok)


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("shift", [300.0, -300.0])
def test_large_logits(F, T, shift):
    # every logit shifted far from 0: the softmax does not change, exponentials
    # without a reference would overflow or vanish
    V, D = 1000, 64
    x, w, y = inputs(T, V, D, "bf16", ignored=None)
    x[:, 0] = 16.0
    w[:, 0] = shift / 16.0
    loss, tok, dx, dw = run(F, x, w, y)
    check(reference(x, w, y), "bf16", D, (V, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, x, w, y, grad=False)
    check(reference(x, w, y), "bf16", D, (V, T), loss, tok)


def test_peaked_and_flat_rows(F):
    # a row that is sure of its target, one that is sure of another, and one
    # that has no preference at all
    V, D = 4000, 128
    x, w, y = inputs(3, V, D, "f16", std=1.0, ignored=None)
    x[0] = (w[y[0]].float() * 2).half()
    x[1] = (w[(y[1] + 1) % V].float() * 2).half()
    x[2] = 0
    loss, tok, dx, dw = run(F, x, w, y)
    check(reference(x, w, y), "f16", D, (V, 3), loss, tok, dx, dw)
    assert abs(float(tok[2]) - math.log(V)) < 1e-5


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", [(5, 1, 64), (130, 1, 8), (6, 3, 40), (200, 2, 64), (150, 700, 128)])
def test_rows_that_are_sure_of_their_target(F, T, V, D, dt):
    """p - 1 at the target, down to probabilities a few 2^-20 from 1 (and one
    column, where it is 0): every probability is good to its logit's error and
    2^-20, whatever is left of the difference."""
    x, w, y = inputs(T, V, D, dt, std=0.05, ignored=None, seed=V)
    lift = torch.linspace(0, 14, T, device=DEV)[:, None]
    toward = w[y].float()
    x = (x.float() * 0.3 + lift * toward / toward.square().sum(1, keepdim=True)).to(DT[dt])
    ref = reference(x, w, y)
    loss, tok, dx, dw = run(F, x, w, y)
    logit = 8 * math.sqrt(D) * 2.0 ** -23 * ref["a"] + 2.0 ** -20
    assert bool(((tok.double() - ref["tok"]).abs() <= logit * (1 + ref["tok"])).all())
    p = torch.softmax(x.double() @ w.double().t(), 1)
    le = float(logit.max())
    for got, want, size, each in ((dx, ref["dx"], ref["sx"], p @ w.double().abs() / ref["n"]),
                                  (dw, ref["dw"], ref["sw"], p.t() @ x.double().abs() / ref["n"])):
        rounding = 4 * math.sqrt(max(V, T)) * 2.0 ** -23 if dt == "f32" else 1.1 * (U[dt] + 2.0 ** -11)
        bound = rounding * size + 2 * le * each + U[dt] * want.abs() + (2.0 ** -25 if dt == "f16" else 1e-37)
        assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [3, 40, 300])
def test_one_column_has_no_gradient(F, T, dt):
    """softmax of one logit is 1 whatever the logit is, its rounding included:
    the exponential and the sum see the same one, so p - 1 is no more than an
    exponential's two units and a division's one on either side, under 2^-21,
    and does not grow with the logit."""
    D = 64
    x, w, _ = inputs(T, 1, D, dt, std=4.0, ignored=None, seed=T)
    y = torch.zeros(T, dtype=torch.int64, device=DEV)
    assert float((x.double() @ w.double().t()).abs().max()) > 30
    _, _, dx, dw = run(F, x, w, y, reduction="sum")
    least = 2.0 ** -25 if dt == "f16" else 1e-37
    d, more = 2.0 ** -21, 1 + 4 * U[dt]
    assert bool((dx.double().abs() <= d * more * w.double().abs() + least).all())
    assert bool((dw.double().abs() <= d * more * x.double().abs().sum(0) + least).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("T", [1, 4, 25, 300])
def test_one_column_has_no_loss(F, T, grad, dt):
    """Exactly none: the only exponential is 1, and so is the sum."""
    x, w, _ = inputs(T, 1, 64, dt, std=4.0, ignored=None, seed=T)
    y = torch.zeros(T, dtype=torch.int64, device=DEV)
    assert bool((run(F, x, w, y, grad=grad)[1] == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("T", [4, 25, 300])
def test_losses_of_rows_that_are_sure_of_their_target(F, T, grad, dt):
    """From about 0.2 down to nothing. A loss is the logarithm of 1 and a few
    small terms: never negative, 0 where they are beyond fp32. Each term is good
    to both logits' errors and 2^-17 (the exponent, below 2^6, is rounded twice
    by 2^-24 of itself), and a row's sum of these 700 takes at most 32 roundings
    of 2^-24 beside the 1: 2^-19."""
    V, D = 700, 128
    x, w, y = inputs(T, V, D, dt, ignored=None, seed=V)
    lift = torch.linspace(8, 40, T, device=DEV)[:, None]
    toward = w[y].float()
    x = (x.float() * 0.05 + lift * toward / toward.square().sum(1, keepdim=True)).to(DT[dt])
    ref = reference(x, w, y)
    tok = run(F, x, w, y, grad=grad)[1]
    assert bool((tok >= 0).all()) and bool((tok[ref["tok"] < 1e-12] == 0).all())
    le = 8 * math.sqrt(D) * 2.0 ** -23 * ref["a"]
    bound = (2 * le + 2.0 ** -17) * ref["tok"] + 2.0 ** -19
    assert bool(((tok.double() - ref["tok"]).abs() <= bound).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [4, 25, 300])
@pytest.mark.parametrize("size", [1e6, 1e10, 1e30])
def test_logits_of_any_finite_size(F, T, size, dt):
    V, D = 700, 64
    x, w, y = inputs(T, V, D, dt, ignored="some")
    x *= size
    ref = reference(x, w, y)
    loss, tok, _, _ = run(F, x, w, y, grad=False)
    check(ref, dt, D, (V, T), loss, tok)
    loss, tok, dx, dw = run(F, x, w, y)
    check(ref, dt, D, (V, T), loss, tok)
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())


def test_gradients_against_differences(F):
    # the loss along a direction, in fp32: (L(x + h d) - L(x - h d)) / 2h = dx . d
    T, V, D = 12, 300, 64
    x, w, y = inputs(T, V, D, "f32", std=0.3)
    _, _, dx, dw = run(F, x, w, y, reduction="sum")
    g = torch.Generator(device=DEV).manual_seed(1)
    # third derivative below 2 |d|^3-ish terms: h = 2^-6 keeps h^2 terms and the
    # losses' own 2^-20 relative error / h both under 2 %
    h = 2.0 ** -6
    for which, grad in (("x", dx), ("w", dw)):
        d = torch.empty_like(grad).normal_(generator=g)
        d /= d.norm()
        moved = [run(F, x + s * h * d if which == "x" else x, w + s * h * d if which == "w" else w, y,
                     grad=False, reduction="sum")[1].double().sum() for s in (1, -1)]
        slope = float(moved[0] - moved[1]) / (2 * h)
        want = float((grad.double() * d.double()).sum())
        assert abs(slope - want) <= 0.02 * float(grad.double().norm()), (slope, want)


def test_same_bits_every_time(F):
    x, w, y = inputs(500, 3000, 256, "bf16", ignored="some")
    a = run(F, x, w, y)
    for _ in range(3):
        b = run(F, x, w, y)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_one_head_for_calls_of_many_sizes_and_streams(F):
    V, D = 1000, 128
    head = F.HeadLoss(V, D, torch.bfloat16, 600)
    s = torch.cuda.Stream()
    for k, T in enumerate((600, 1, 37, 256, 8, 599)):
        x, w, y = inputs(T, V, D, "bf16", seed=k)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        s.wait_stream(torch.cuda.current_stream())
        loss, tok = head.forward_backward(x, w, y, dx, dw, stream=s)
        l2, t2 = head.forward(x, w, y, stream=s)
        s.synchronize()
        ref = reference(x, w, y)
        check(ref, "bf16", D, (V, T), loss, tok, dx, dw)
        check(ref, "bf16", D, (V, T), l2, t2)


def block_with_a_queued_reader(nbytes):
    """A copy, still to be made on the current stream, of a block of that many
    bytes, which is already back with the allocator."""
    block = torch.full((nbytes,), 7, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    return block.clone()


@pytest.mark.parametrize("form", ["function", "object", "growth"])
def test_a_workspace_waits_for_its_memorys_last_user(F, form):
    from sharded_fsdp_reduce_gb300 import loss as mod
    T, V, D = 300, 5000, 256
    x, w, y = inputs(T, V, D, "bf16")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    loss, tok = torch.empty((), device=DEV), torch.empty(T, device=DEV)
    s = torch.cuda.Stream()
    if form == "growth":  # the weight at an address that has to be packed
        head = F.HeadLoss(V, D, torch.bfloat16, T)
        buf = torch.empty(V * D + 1, dtype=torch.bfloat16, device=DEV)
        buf[1:].view(V, D).copy_(w)
        w = buf[1:].view(V, D)
    F.fsdp_head_loss(x, w, y, loss, tok, dx, dw)  # (a kernel's first launch waits for the device)
    need = mod._workspace_bytes(mod._args(x, w, y, loss, tok, dx, dw, IGNORE, "mean", 1.0, 0, None))
    assert need > 4 << 20
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    copy = block_with_a_queued_reader(need + 1024)
    if form == "function":
        F.fsdp_head_loss(x, w, y, loss, tok, dx, dw, stream=s)
    else:
        if form == "object":
            head = F.HeadLoss(V, D, torch.bfloat16, T)
        head.forward_backward(x, w, y, dx, dw, loss=loss, token_loss=tok, stream=s)
    torch.cuda.synchronize()
    assert bool((copy == 7).all())
    check(reference(x, w, y), "bf16", D, (V, T), loss, tok, dx, dw)


def test_workspace_grows_for_packed_operands(F):
    V, D, T = 700, 72, 50
    head = F.HeadLoss(V, D, torch.bfloat16, T)
    x, w, y = inputs(T, V, D, "bf16")
    buf = torch.empty(V * D + 1, dtype=torch.bfloat16, device=DEV)
    w1 = buf[1:].view(V, D)
    w1.copy_(w)
    a, b = torch.empty_like(w), torch.empty_like(w)
    head.forward_backward(x, w, y, None, a)
    head.forward_backward(x, w1, y, None, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dt,most,V,D", [("bf16", 600, 2000, 1024), ("f16", 1100, 4000, 1024), ("f32", 1100, 1003, 512),
                                         ("f16", 300, 300, 65)])
@pytest.mark.parametrize("grad", [True, False])
def test_no_shorter_call_grows_the_workspace(F, dt, most, V, D, grad):
    head = F.HeadLoss(V, D, DT[dt], most, grad=grad)
    at, size = head._ws_at, head._ws_bytes
    x, w, y = inputs(most, V, D, dt, ignored="some")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    # (1024 and 585 rows cut a product into more pieces than 1100 and 600)
    lengths = (1100, 1025, 1024, 1000, 700, 600, 585, 513, 512, 300, 257, 256, 255, 130, 65, 64, 33, 25, 24, 9, 8, 5, 4, 1)
    for T in (t for t in lengths if t <= most):
        if grad:
            head.forward_backward(x[:T], w, y[:T], dx[:T], dw)
            head.forward_backward(x[:T], w, y[:T], None, dw)
            head.forward_backward(x[:T], w, y[:T], dx[:T], None)
        head.forward(x[:T], w, y[:T])
        assert (head._ws_at, head._ws_bytes) == (at, size), T


def test_a_captured_graph_outlives_a_growth(F):
    """A graph's calls keep writing to the workspace that they were captured
    with: it has to stay theirs when a later call takes a larger one."""
    T, V, D = 64, 5000, 256
    x, w, y = inputs(T, V, D, "bf16", ignored="some")
    head = F.HeadLoss(V, D, torch.bfloat16, T)
    size = head._ws_bytes
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    loss, tok = torch.empty((), device=DEV), torch.empty(T, device=DEV)
    head.forward_backward(x, w, y, dx, dw, loss=loss, token_loss=tok)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        head.forward_backward(x, w, y, dx, dw, loss=loss, token_loss=tok)
    buf = torch.empty(V * D + 1, dtype=torch.bfloat16, device=DEV)
    buf[1:].view(V, D).copy_(w)
    for _ in range(2):
        head.forward_backward(x, buf[1:].view(V, D), y, None, torch.empty_like(w))
    assert head._ws_bytes > size
    torch.cuda.synchronize()
    others = [torch.full((size + 1024,), 7, dtype=torch.uint8, device=DEV) for _ in range(3)]
    for t in (dx, dw, loss, tok):
        t.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    check(reference(x, w, y), "bf16", D, (V, T), loss, tok, dx, dw)
    assert all(bool((o == 7).all()) for o in others)


def test_captured_in_a_graph(F):
    T, V, D = 200, 1200, 128
    x, w, y = inputs(T, V, D, "bf16")
    head = F.HeadLoss(V, D, torch.bfloat16, T)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    loss, tok = torch.empty((), device=DEV), torch.empty(T, device=DEV)
    head.forward_backward(x, w, y, dx, dw, loss=loss, token_loss=tok)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        head.forward_backward(x, w, y, dx, dw, loss=loss, token_loss=tok)
    for k in range(2):
        x2, w2, y2 = inputs(T, V, D, "bf16", seed=30 + k, ignored="some")
        x.copy_(x2), w.copy_(w2), y.copy_(y2)
        g.replay()
        torch.cuda.synchronize()
        check(reference(x, w, y), "bf16", D, (V, T), loss, tok, dx, dw)


def test_made_within_a_capture_and_used_outside_it(F):
    T, V, D = 200, 1200, 128
    x, w, y = inputs(T, V, D, "bf16")
    loss, tok = torch.empty((), device=DEV), torch.empty(T, device=DEV)
    run(F, x, w, y, grad=False)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        head = F.HeadLoss(V, D, torch.bfloat16, T)
        head.forward(x, w, y, loss=loss, token_loss=tok)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    l2, t2 = head.forward_backward(x, w, y, dx, dw)
    g.replay()
    torch.cuda.synchronize()
    ref = reference(x, w, y)
    check(ref, "bf16", D, (V, T), loss, tok)
    check(ref, "bf16", D, (V, T), l2, t2, dx, dw)


def test_results_longer_than_32_bits_of_elements(F):
    # the exponentials of one band pass 2^31 elements
    T, V, D = 16400, 131100, 8
    x, w, y = inputs(T, V, D, "bf16", std=0.3, ignored=None)
    loss, tok, dx, dw = run(F, x, w, y, band=T)
    at = torch.tensor([0, 1, 8191, 16383, 16384, T - 1], device=DEV)
    ref = reference(x[at], w, y[at], "sum")
    logit = 8 * math.sqrt(D) * 2.0 ** -23 * ref["a"]
    assert bool(((tok[at].double() - ref["tok"]).abs() <= logit + 2.0 ** -20 * ref["lse"]).all())
    bound = 1.1 * (U["bf16"] + 2.0 ** -11) * ref["sx"] + U["bf16"] * ref["dx"].abs()
    assert bool(((dx[at].double() * T - ref["dx"]).abs() <= bound + 1e-30).all())
    del dx
    # the last vocabulary rows' gradient, from the definition
    lse = torch.cat([torch.logsumexp(x[i:i + 2048].double() @ w.double().t(), 1) for i in range(0, T, 2048)])
    cols = torch.arange(V - 5, V, device=DEV)
    p = torch.exp(x.double() @ w[cols].double().t() - lse[:, None])
    p -= (y[:, None] == cols[None, :]).double()
    want = p.t() @ x.double() / T
    size = p.abs().t() @ x.double().abs() / T
    assert bool(((dw[cols].double() - want).abs() <= 1.1 * (U["bf16"] + 2.0 ** -11) * size
                 + U["bf16"] * want.abs()).all())


def test_refusals(F):
    x, w, y = inputs(20, 100, 64, "bf16")
    head = F.HeadLoss(100, 64, torch.bfloat16, 20)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for bad in (
        lambda: head.forward(x.float(), w, y),
        lambda: head.forward(x, w[:50], y),
        lambda: head.forward(torch.cat([x, x]), w, y),
        lambda: head.forward(x[:, :32], w, y),
        lambda: head.forward(x, w, y[:10]),
        lambda: head.forward(x, w, y.int()),
        lambda: head.forward(x, w, y.cpu()),
        lambda: head.forward(x.t().contiguous().t(), w, y),
        lambda: head.forward(x[:1].expand(20, 64), w, y),
        lambda: head.forward_backward(x, w, y, dx.float(), dw),
        lambda: head.forward_backward(x, w, y, dx, dw[:99]),
        lambda: head.forward(x, w, y, loss=torch.empty(2, device=DEV)),
        lambda: F.HeadLoss(100, 64, torch.bfloat16, 20, reduction="none"),
    ):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(TypeError):
        F.HeadLoss(100, 64, torch.float64, 20)
    for bad in (
        lambda: head.forward_backward(x, w, y, x, dw),                       # a gradient over its input
        lambda: head.forward_backward(x, w, y, dx, w),
        lambda: head.forward_backward(x, w, y, dw[:20], dw),                 # two gradients in one place
        lambda: head.forward_backward(x, w, y, dx, dw, grad_scale=float("nan")),
        lambda: F.HeadLoss(100, 64, torch.bfloat16, 20, band=-1),
    ):
        with pytest.raises(F.FsdpError):
            bad()


def test_a_workspace_too_small_is_refused(F):
    import ctypes
    from sharded_fsdp_reduce_gb300 import _lib, loss as mod
    x, w, y = inputs(20, 100, 64, "bf16")
    out = torch.empty((), device=DEV)
    a = mod._args(x, w, y, out, None, None, None, IGNORE, "mean", 1.0, 0, None)
    need = mod._workspace_bytes(a)
    ws = mod._workspace(need, x.device)
    lib = _lib.load()
    assert lib.fsdp_head_loss(ctypes.byref(a), ws.data_ptr(), need - 1, None) == _lib.FSDP_ERR_INVALID_ARG
    assert lib.fsdp_head_loss(ctypes.byref(a), ws.data_ptr() + 16, need, None) == _lib.FSDP_ERR_ALIGNMENT
    assert lib.fsdp_head_loss(ctypes.byref(a), None, need, None) == _lib.FSDP_ERR_INVALID_ARG


def test_a_bounded_wait_has_one_outcome_per_warp(F):
    """The products' waits, without a fault: an arrival that never comes runs
    out and is counted, one in time is seen, and one that comes as the limit
    passes has the same outcome in all lanes of a warp."""
    out = torch.empty(128, dtype=torch.int32, device=DEV)
    waits = torch.zeros(1, dtype=torch.int32, device=DEV)

    def check_wait(limit, arrive):
        waits.zero_()
        F.fsdp_check_head_loss_wait(limit, arrive, out, waits)
        torch.cuda.synchronize()
        warps = out.reshape(4, 32)
        assert bool((warps == warps[:, :1]).all()), (limit, arrive, warps.tolist())
        gave_up = int((warps[:, 0] == 0).sum())
        assert (1 if gave_up else 0) <= int(waits) <= gave_up
        return gave_up

    assert check_wait(1 << 20, -1) == 4
    assert check_wait(1 << 20, 1000) == 0
    for k in range(200):
        limit = 2000 + 97 * k
        check_wait(limit, limit + 13 * (k % 41) - 250)
    with pytest.raises(F.FsdpError):
        F.fsdp_check_head_loss_wait(0, 10, out)
    with pytest.raises(F.FsdpError):
        F.fsdp_check_head_loss_wait(10, (1 << 31) + 1, out)
    with pytest.raises(ValueError):
        F.fsdp_check_head_loss_wait(10, 10, out[:64])
    # the context still works
    x, w, y = inputs(40, 300, 64, "bf16")
    loss, tok, dx, dw = run(F, x, w, y)
    check(reference(x, w, y), "bf16", 64, (300, 40), loss, tok, dx, dw)
