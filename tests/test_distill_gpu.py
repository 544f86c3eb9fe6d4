"""The distillation loss (fsdp_head_distill, HeadDistill) against its definition
in fp64.

Tolerances, derived from the operations (u = 2^-8 bf16, 2^-11 fp16 unit
roundoff; A = max_v sum_k |x_k w_k| of a row; s a row's entries):
* a logit: fp32 products and sums, le = 8 sqrt(D) 2^-23 A; the student's log
  probability of an entry has two of them over the temperature, 2^-20 max(1,
  |lse|) for the exponentials and sums behind lse, and the roundings of a
  difference and a product, 2^-22 of itself.
* the teacher's: 2^-22 (1 + |log p|) for a difference, a product and an
  exponential, and c = (s / 32 + 8) 2^-24 + 2^-21 for the sum of s exponentials
  and its logarithm; as much again relative for p.
* a token's loss: the sum over its entries of p times both errors, and of p's
  error times the term; its own sum (s / 32 + 8) 2^-24 of the magnitudes.
* a gradient element: sums of errors of d times |w| (or |x|): q's error and p's;
  for 16-bit types d's rounding u and the exponential's 2^-11, but 2^-40 of the
  largest of its 64 columns where it is small against that; 10 % for
  second-order terms; and the output's own rounding. fp32 heads: the split
  products and sums 4 sqrt(K) 2^-23, the output 2^-23.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
INF = float("inf")


@pytest.fixture(scope="module")
def F():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sharded_fsdp_reduce_gb300 as F
    return F


def inputs(T, V, D, K, dt, seed=0, std=0.05, kind="some", teacher=torch.float32, ids=torch.int64, spread=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(T, D, device=DEV).normal_(generator=g).to(DT[dt])
    w = (torch.empty(V, D, device=DEV).normal_(generator=g) * std).to(DT[dt])
    a = torch.empty(T, K, device=DEV).normal_(generator=g) * spread
    if kind == "twice" or K > V:  # tokens named more than once
        i = torch.randint(0, max(1, min(V, K // 2 + 1)), (T, K), device=DEV, generator=g) * max(1, V // (K // 2 + 1))
        i.clamp_(max=V - 1)
    else:
        i = torch.stack([torch.randperm(V, device=DEV, generator=g)[:K] for _ in range(min(T, 64))])
        i = i.repeat(-(-T // 64), 1)[:T]
        i = (i + torch.arange(T, device=DEV)[:, None] * 7) % V
    if kind == "some":  # fewer entries, none, and minus infinities
        i[torch.rand(T, K, device=DEV, generator=g) < 0.2] = -1
        a[torch.rand(T, K, device=DEV, generator=g) < 0.1] = -INF
        none = torch.rand(T, device=DEV, generator=g) < 0.2
        i[none] = -1
        a[none] = float("nan")  # what lies in unused entries does not matter
    elif kind == "none":
        i[:] = -1
    return x, w, a.to(teacher), i.to(ids)


def reference(x, w, a, i, tau=1.0, reduction="mean", grad_scale=1.0):
    """Loss, row losses, gradients and their error bounds' parts, in fp64."""
    stored16 = x.dtype != torch.float32
    x, w, i = x.double(), w.double(), i.long()
    T, K = i.shape
    live = (i != -1) & (a.double() != -INF)
    valid = live.any(1)
    z = (x @ w.t())
    lse = torch.logsumexp(z / tau, 1)
    logq = z / tau - lse[:, None]
    t = torch.where(live, a.double() / tau, -INF)
    t[~valid] = 0.0
    logp = torch.where(live, t - torch.logsumexp(t, 1)[:, None], 0.0)
    p = torch.where(live, torch.exp(logp), 0.0)
    lq = torch.where(live, logq.gather(1, torch.where(live, i, 0)), 0.0)
    term = torch.where(p > 0, logp - lq, 0.0)
    tok = torch.where(valid, tau * tau * (p * term).sum(1), 0.0)
    n = max(int(valid.sum()), 1) if reduction == "mean" else 1
    g = grad_scale * tau / n
    A = (x.abs() @ w.abs().t()).amax(1)
    le = 8 * math.sqrt(x.shape[1]) * 2.0 ** -23 * A
    c = (K / 32 + 8) * 2.0 ** -24 + 2.0 ** -21
    dq = 2 * le / tau + 2.0 ** -20 * lse.abs().clamp(min=1)      # of log q, but for 2^-22 of itself
    dp = 2.0 ** -22 * (1 + logp.abs()) + c                      # of log p, and relative of p
    size = term.abs()
    tol = tau * tau * (p * (dq[:, None] + 2.0 ** -22 * lq.abs() + dp * (1 + size))).sum(1)
    tol += tau * tau * (K / 32 + 8) * 2.0 ** -24 * (p * size).sum(1)
    q = torch.exp(logq)
    d = q.clone().scatter_add_(1, torch.where(live, i, 0), -p)
    # 16-bit heads: an exponential is an fp16 number times 2^-15 of the largest
    # of its 64 columns, at half a subnormal step 2^-25 2^-15 off
    least = torch.nn.functional.pad(q, (0, -q.shape[1] % 64)).view(T, -1, 64).amax(2).repeat_interleave(64, 1)
    least = least[:, :q.shape[1]] * (2.0 ** -40 if stored16 else 0.0)
    ed = (q * (dq[:, None] + 2.0 ** -20) + least).scatter_add_(1, torch.where(live, i, 0), p * dp)
    d *= valid[:, None]
    ed *= valid[:, None]
    out = dict(loss=tok.sum() / n, tok=tok, tol=tol * valid + 1e-38, n=n, valid=valid)
    for name, m in (("x", w), ("w", x)):
        of = (lambda d: d @ m) if name == "x" else (lambda d: d.t() @ m)
        size = (lambda d: d @ m.abs()) if name == "x" else (lambda d: d.t() @ m.abs())
        out["d" + name], out["s" + name], out["e" + name] = g * of(d), abs(g) * size(d.abs()), abs(g) * size(ed)
    return out


def check(ref, dt, K, loss, tok, dx=None, dw=None):
    err = (tok.double() - ref["tok"]).abs()
    over = err > ref["tol"] * 1.1
    assert not bool(over.any()), f"row loss off by {float((err / ref['tol']).max()):.3g} of what is allowed"
    assert bool((tok[~ref["valid"]] == 0).all())
    total = float(ref["tol"].sum()) * 1.1 / ref["n"]
    assert abs(float(loss) - float(ref["loss"])) <= total + 2.0 ** -23 * abs(float(ref["loss"]))
    for got, name, k in ((dx, "x", K[0]), (dw, "w", K[1])):
        if got is None:
            continue
        want, size, e = ref["d" + name], ref["s" + name], ref["e" + name]
        if dt == "f32":
            bound = 1.1 * (e + 4 * math.sqrt(k) * 2.0 ** -23 * size) + 2.0 ** -23 * want.abs() + 1e-37
        else:
            bound = 1.1 * ((U[dt] + 2.0 ** -11) * size + e) + U[dt] * want.abs()
            bound += 2.0 ** -25 if dt == "f16" else 1e-37  # half the smallest subnormal step
        err = (got.double() - want).abs()
        over = err > bound
        assert not bool(over.any()), (f"d{name}: {int(over.sum())} of {over.numel()} beyond the bound, first at "
                                      f"{over.nonzero()[0].tolist()}, worst ratio {float((err / bound).max()):.3g}")


def run(F, x, w, a, i, grad=True, tau=1.0, **kw):
    T, V = x.shape[0], w.shape[0]
    head = F.HeadDistill(V, w.shape[1], x.dtype, T, i.shape[1], temperature=tau, grad=grad,
                         reduction=kw.pop("reduction", "mean"), band=kw.pop("band", 0))
    waits = torch.zeros(1, dtype=torch.int32, device=DEV)
    if not grad:
        loss, tok = head.forward(x, w, a, i, wait_timeouts=waits)
        dx = dw = None
    else:
        dx, dw = kw.pop("dx", None), kw.pop("dw", None)
        dx = torch.full_like(x, float("nan")) if dx is None else dx
        dw = torch.full_like(w, float("nan")) if dw is None else dw
        loss, tok = head.forward_backward(x, w, a, i, dx, dw, wait_timeouts=waits, **kw)
    torch.cuda.synchronize()
    assert int(waits.item()) == 0
    return loss, tok, dx, dw


SIZES = [  # tokens, vocab, dim, entries: tiles' edges, odd ones, one of everything, more entries than columns
    (1, 1, 8, 1), (1, 1000, 64, 5), (2, 257, 72, 64), (5, 3, 16, 9), (31, 128, 128, 33), (33, 129, 8, 1), (128, 256, 64, 100),
    (129, 1003, 200, 17), (255, 511, 264, 65), (257, 640, 512, 129), (300, 5000, 768, 256), (1021, 3001, 320, 31),
    (70, 2000, 64, 1024), (130, 1500, 96, 513),
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D,K", SIZES)
def test_losses(F, T, V, D, K, dt):
    for kind in ("some", "twice"):
        x, w, a, i = inputs(T, V, D, K, dt, kind=kind)
        loss, tok, _, _ = run(F, x, w, a, i, grad=False)
        check(reference(x, w, a, i), dt, (V, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D,K", SIZES)
def test_gradients(F, T, V, D, K, dt):
    for kind in ("some", "twice"):
        x, w, a, i = inputs(T, V, D, K, dt, kind=kind, seed=1)
        loss, tok, dx, dw = run(F, x, w, a, i)
        check(reference(x, w, a, i), dt, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 17, 24, 25])
@pytest.mark.parametrize("V,D,K", [(5003, 768, 50), (129, 100, 7), (33, 3, 33)])
def test_a_few_rows(F, T, V, D, K, dt):
    x, w, a, i = inputs(T, V, D, K, dt, seed=T, kind="some" if T > 4 else "all")
    ref = reference(x, w, a, i)
    loss, tok, _, _ = run(F, x, w, a, i, grad=False)
    check(ref, dt, (V, T), loss, tok)
    loss, tok, dx, dw = run(F, x, w, a, i)
    check(ref, dt, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tau", [0.25, 0.7, 2.0, 10.0])
@pytest.mark.parametrize("T", [3, 200])
def test_temperatures(F, T, tau, dt):
    x, w, a, i = inputs(T, 1500, 96, 40, dt, seed=2, spread=4.0)
    ref = reference(x, w, a, i, tau)
    loss, tok, dx, dw = run(F, x, w, a, i, tau=tau)
    check(ref, dt, (1500, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, x, w, a, i, tau=tau, grad=False)
    check(ref, dt, (1500, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,tau", [(4, 0.5), (4, 0.05), (150, 0.5), (150, 0.05)])
def test_probabilities_far_apart(F, T, tau, dt):
    # logits over the temperature up to 100 apart: columns at 2^-40 of their
    # neighbours and less
    x, w, a, i = inputs(T, 3001, 264, 5, dt, seed=8, std=0.15 if tau == 0.5 else 0.05, kind="all")
    ref = reference(x, w, a, i, tau)
    loss, tok, dx, dw = run(F, x, w, a, i, tau=tau)
    check(ref, dt, (3001, T), loss, tok, dx, dw)


@pytest.mark.parametrize("teacher", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("T", [4, 150])
def test_types_of_the_teacher(F, T, ids, teacher):
    x, w, a, i = inputs(T, 900, 64, 30, "bf16", teacher=DT[teacher], ids=ids, seed=3)
    loss, tok, dx, dw = run(F, x, w, a, i)
    check(reference(x, w, a, i), "bf16", (900, T), loss, tok, dx, dw)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,band", [(700, 256), (513, 512), (300, 100), (9, 1)])
def test_bands_of_tokens(F, T, band, dt):
    V, D, K = 777, 200, 20
    x, w, a, i = inputs(T, V, D, K, dt, seed=7)
    ref = reference(x, w, a, i, 2.0)
    loss, tok, dx, dw = run(F, x, w, a, i, band=band, tau=2.0)
    check(ref, dt, (V, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, x, w, a, i, grad=False, band=band, tau=2.0)
    check(ref, dt, (V, T), loss, tok)


@pytest.mark.parametrize("dt,scale", [("bf16", 1.0), ("f16", 256.0), ("f32", 0.125)])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_reduction_and_loss_scale(F, dt, scale, reduction):
    T, V, D, K = 90, 1500, 96, 12
    if dt == "f16" and reduction == "sum":
        scale = 4.0  # the gradients have to fit fp16
    x, w, a, i = inputs(T, V, D, K, dt, seed=9)
    loss, tok, dx, dw = run(F, x, w, a, i, tau=2.0, reduction=reduction, grad_scale=scale)
    check(reference(x, w, a, i, 2.0, reduction, scale), dt, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off,pad", [(0, 8), (8, 24), (1, 0), (3, 5), (2, 6)])
def test_views_at_any_offset_and_stride(F, off, pad, dt):
    T, V, D, K = 140, 700, 136, 24
    x0, w0, a0, i0 = inputs(T, V, D, K, dt, seed=6)

    def place(rows, cols, dtype, src=None):
        buf = torch.full((off + rows * (cols + pad) + 64,), 7, dtype=dtype, device=DEV)
        v = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        if src is not None:
            v.copy_(src)
        return buf, v

    x, w = place(T, D, DT[dt], x0)[1], place(V, D, DT[dt], w0)[1]
    a, i = place(T, K, torch.float32, a0)[1], place(T, K, torch.int64, i0)[1]
    bx, dx = place(T, D, DT[dt])
    bw, dw = place(V, D, DT[dt])
    ref = reference(x0, w0, a0, i0)
    loss, tok, _, _ = run(F, x, w, a, i, dx=dx, dw=dw)
    check(ref, dt, (V, T), loss, tok, dx, dw)
    for buf, v, rows in ((bx, dx, T), (bw, dw, V)):  # nothing beside the gradients is written
        v.zero_()
        assert int((buf == 7).sum()) == buf.numel() - rows * D
    loss, tok, _, _ = run(F, x, w, a, i, grad=False)
    check(ref, dt, (V, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 200])
def test_no_row_counts(F, T, dt):
    x, w, a, i = inputs(T, 600, 64, 10, dt, kind="none")
    x[:] = float("nan")
    loss, tok, dx, dw = run(F, x, w, a, i)
    assert float(loss) == 0.0 and not bool(tok.any()) and not bool(dx.any()) and not bool(dw.any())
    assert float(run(F, x, w, a, i, grad=False)[0]) == 0.0
    # entries without any probability do not count either
    x, w, a, i = inputs(T, 600, 64, 10, dt, kind="all")
    a[:] = -INF
    loss, tok, dx, dw = run(F, x, w, a, i)
    assert float(loss) == 0.0 and not bool(tok.any()) and not bool(dx.any()) and not bool(dw.any())


def test_no_tokens(F):
    x, w, a, i = inputs(1, 100, 64, 4, "bf16")
    loss, tok, dx, dw = run(F, x[:0], w, a[:0], i[:0])
    assert float(loss) == 0.0 and tok.numel() == 0 and not bool(dw.any())


def test_either_gradient_alone(F):
    x, w, a, i = inputs(150, 900, 128, 20, "bf16")
    head = F.HeadDistill(900, 128, torch.bfloat16, 150, 20)
    both = [torch.empty_like(x), torch.empty_like(w)]
    head.forward_backward(x, w, a, i, *both)
    one, two = torch.empty_like(x), torch.empty_like(w)
    head.forward_backward(x, w, a, i, one, None)
    head.forward_backward(x, w, a, i, None, two)
    assert torch.equal(one, both[0]) and torch.equal(two, both[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [4, 300])
def test_the_order_of_the_entries_does_not_matter(F, T, dt):
    """Beyond the roundings of the teacher's sum, which is taken as they come in."""
    x, w, a, i = inputs(T, 800, 64, 50, dt, kind="some", seed=4)
    order = torch.randperm(50, device=DEV)
    one = run(F, x, w, a, i)
    two = run(F, x, w, a[:, order].contiguous(), i[:, order].contiguous())
    three = run(F, x, w, a, i)
    assert all(torch.equal(p, q) for p, q in zip(one, three))
    ref = reference(x, w, a, i)
    for r in (one, two):
        check(ref, dt, (800, T), *r)


@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_wrong_entries_show_as_nan(F, T, dt):
    V, D, K = 500, 64, 8
    for what in (V, -2, 2 ** 40, "nan", "inf"):
        x, w, a, i = inputs(T, V, D, K, dt, kind="all")
        good = run(F, x, w, a, i)[1]
        if isinstance(what, str):
            a[2, 3] = float(what)
        else:
            i[2, 3] = what
        loss, tok, dx, dw = run(F, x, w, a, i)
        assert math.isnan(float(loss)) and math.isnan(float(tok[2])) and bool(torch.isnan(dx[2]).all())
        keep = torch.arange(T, device=DEV) != 2
        assert torch.equal(tok[keep], good[keep])
        assert not bool(torch.isnan(dx[keep]).any()) and bool(torch.isnan(dw).all())
        assert math.isnan(float(run(F, x, w, a, i, grad=False)[0]))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [4, 8, 24, 25, 300])
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
def test_a_counted_row_that_is_not_finite(F, T, bad, dt):
    V, D = 500, 64
    x, w, a, i = inputs(T, V, D, 9, dt, kind="all")
    good = run(F, x, w, a, i, grad=False)[1]
    x[3, 5] = bad
    keep = torch.arange(T, device=DEV) != 3
    loss, tok, _, _ = run(F, x, w, a, i, grad=False)
    assert math.isnan(float(loss)) and math.isnan(float(tok[3])) and torch.equal(tok[keep], good[keep])
    loss, tok, dx, dw = run(F, x, w, a, i)
    assert math.isnan(float(tok[3])) and bool(torch.isnan(dx[3]).all()) and bool(torch.isnan(dw).all())
    assert not bool(torch.isnan(dx[keep]).any()) and not bool(torch.isnan(tok[keep]).any())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,band", [(3, 0), (64, 0), (300, 0), (600, 256)])
def test_what_lies_in_rows_without_entries_does_not_matter(F, T, band, dt):
    V, D, K = 700, 136, 11
    x, w, a, i = inputs(T, V, D, K, dt, seed=3)
    i[0] = torch.arange(K, device=DEV) * 60
    a[0] = 1.0
    i[1] = -1
    ref = reference(x, w, a, i)
    dirty = x.clone()
    junk = torch.tensor([float("nan"), INF, -INF, 6e4], device=DEV).to(DT[dt])
    dirty[~ref["valid"]] = junk.repeat(D // 4)
    loss, tok, dx, dw = run(F, dirty, w, a, i, band=band)
    check(ref, dt, (V, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, dirty, w, a, i, grad=False, band=band)
    check(ref, dt, (V, T), loss, tok)


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_columns_that_cannot_be_drawn(F, T, dt):
    """Logits of minus infinity (a masked part of the vocabulary, whole spans of
    it): nothing where the teacher gives them nothing; an infinite loss where it
    does."""
    V, D, K = 900, 64, 10
    x, w, a, i = inputs(T, V, D, K, dt, kind="all")
    x = x.abs() + 0.1
    i %= 100
    w[300:850] = -INF
    keep = torch.cat([torch.arange(300), torch.arange(850, V)]).to(DEV)
    loss, tok, _, _ = run(F, x, w, a, i, grad=False)
    check(reference(x, w[keep], a, i), dt, (V, T), loss, tok)
    i[1, 4] = 400
    tok = run(F, x, w, a, i, grad=False)[1]
    assert float(tok[1]) == INF and int(torch.isinf(tok).sum()) == 1


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("shift", [300.0, -300.0])
def test_large_logits(F, T, shift):
    V, D, K = 1000, 64, 16
    x, w, a, i = inputs(T, V, D, K, "bf16", kind="all")
    x[:, 0] = 16.0
    w[:, 0] = shift / 16.0
    a = a + 1e4  # the teacher's too: only differences matter, of what fp32 keeps of it
    ref = reference(x, w, a, i)
    loss, tok, dx, dw = run(F, x, w, a, i)
    check(ref, "bf16", (V, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, x, w, a, i, grad=False)
    check(ref, "bf16", (V, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [4, 40])
def test_a_student_that_agrees_loses_nothing(F, T, dt):
    """All columns are entries and the teacher's logits are the student's: the
    loss and the gradients are what the roundings leave."""
    V, D = 60, 32
    x, w, _, _ = inputs(T, V, D, 1, dt)
    a = (x.double() @ w.double().t()).float()
    i = torch.arange(V, device=DEV).repeat(T, 1)
    ref = reference(x, w, a, i, 2.0)
    assert float(ref["tok"].abs().max()) < 1e-9
    loss, tok, dx, dw = run(F, x, w, a, i, tau=2.0)
    check(ref, dt, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("T", [3, 130])
def test_one_entry_is_the_cross_entropy(F, T):
    """A teacher that is sure of one token: p = 1, the loss is the cross entropy's
    and the gradients have its bits (the same logits, statistics and sums)."""
    V, D = 700, 64
    x, w, a, i = inputs(T, V, D, 1, "bf16", kind="all")
    y = i[:, 0].contiguous()
    loss, tok, dx, dw = run(F, x, w, a, i)
    l2, t2 = F.HeadLoss(V, D, torch.bfloat16, T).forward(x, w, y)
    # one order of the same terms or another: 2^-22 of them
    z = (x.double() @ w.double().t()).abs().amax(1)
    assert bool(((tok - t2).abs().double() <= 2.0 ** -21 * (z + t2.double() + 1)).all())
    ex, ew = torch.empty_like(x), torch.empty_like(w)
    F.HeadLoss(V, D, torch.bfloat16, T).forward_backward(x, w, y, ex, ew)
    assert torch.equal(dx, ex) and torch.equal(dw, ew)


def test_gradients_against_differences(F):
    T, V, D, K = 12, 300, 64, 7
    x, w, a, i = inputs(T, V, D, K, "f32", std=0.3, kind="twice")
    tau = 2.0
    _, _, dx, dw = run(F, x, w, a, i, reduction="sum", tau=tau)
    g = torch.Generator(device=DEV).manual_seed(1)
    # (L(x + h d) - L(x - h d)) / 2h: h^2 times a third derivative and the
    # losses' own 2^-20 relative error / h both stay under 2 % of the gradient
    h = 2.0 ** -6
    for which, grad in (("x", dx), ("w", dw)):
        d = torch.empty_like(grad).normal_(generator=g)
        d /= d.norm()
        moved = [run(F, x + s * h * d if which == "x" else x, w + s * h * d if which == "w" else w, a, i,
                     grad=False, reduction="sum", tau=tau)[1].double().sum() for s in (1, -1)]
        slope = float(moved[0] - moved[1]) / (2 * h)
        want = float((grad.double() * d.double()).sum())
        assert abs(slope - want) <= 0.02 * float(grad.double().norm()), (slope, want)


def test_same_bits_every_time(F):
    x, w, a, i = inputs(500, 3000, 256, 60, "bf16", kind="twice")
    one = run(F, x, w, a, i)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(one, run(F, x, w, a, i)))


def test_one_head_for_calls_of_many_sizes_and_streams(F):
    V, D, K = 1000, 128, 50
    head = F.HeadDistill(V, D, torch.bfloat16, 600, K, temperature=2.0)
    at, size = head._ws_at, head._ws_bytes
    s = torch.cuda.Stream()
    for n, (T, k) in enumerate(((600, 50), (1, 50), (37, 3), (256, 1), (8, 49), (4, 50), (599, 50))):
        x, w, a, i = inputs(T, V, D, k, "bf16", seed=n)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        s.wait_stream(torch.cuda.current_stream())
        loss, tok = head.forward_backward(x, w, a, i, dx, dw, stream=s)
        l2, t2 = head.forward(x, w, a, i, stream=s)
        s.synchronize()
        ref = reference(x, w, a, i, 2.0)
        check(ref, "bf16", (V, T), loss, tok, dx, dw)
        check(ref, "bf16", (V, T), l2, t2)
        assert (head._ws_at, head._ws_bytes) == (at, size)


def test_workspace_grows_for_packed_operands(F):
    V, D, T, K = 700, 72, 50, 9
    head = F.HeadDistill(V, D, torch.bfloat16, T, K)
    x, w, a, i = inputs(T, V, D, K, "bf16")
    buf = torch.empty(V * D + 1, dtype=torch.bfloat16, device=DEV)
    w1 = buf[1:].view(V, D)
    w1.copy_(w)
    p, q = torch.empty_like(w), torch.empty_like(w)
    head.forward_backward(x, w, a, i, None, p)
    head.forward_backward(x, w1, a, i, None, q)
    assert torch.equal(p, q)


@pytest.mark.parametrize("T", [4, 200])
def test_captured_in_a_graph(F, T):
    V, D, K = 1200, 128, 20
    x, w, a, i = inputs(T, V, D, K, "bf16")
    head = F.HeadDistill(V, D, torch.bfloat16, T, K)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    loss, tok = torch.empty((), device=DEV), torch.empty(T, device=DEV)
    head.forward_backward(x, w, a, i, dx, dw, loss=loss, token_loss=tok)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        head.forward_backward(x, w, a, i, dx, dw, loss=loss, token_loss=tok)
    for k in range(2):
        x2, w2, a2, i2 = inputs(T, V, D, K, "bf16", seed=30 + k)
        x.copy_(x2), w.copy_(w2), a.copy_(a2), i.copy_(i2)
        g.replay()
        torch.cuda.synchronize()
        check(reference(x, w, a, i), "bf16", (V, T), loss, tok, dx, dw)


def test_refusals(F):
    x, w, a, i = inputs(20, 100, 64, 5, "bf16")
    head = F.HeadDistill(100, 64, torch.bfloat16, 20, 5)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for bad in (
        lambda: head.forward(x.float(), w, a, i),
        lambda: head.forward(x, w[:50], a, i),
        lambda: head.forward(torch.cat([x, x]), w, a, i),
        lambda: head.forward(x, w, a[:10], i),
        lambda: head.forward(x, w, a[:, :4], i),
        lambda: head.forward(x, w, a, i[:10]),
        lambda: head.forward(x, w, a, i.short()),
        lambda: head.forward(x, w, a, i.cpu()),
        lambda: head.forward(x, w, a.cpu(), i),
        lambda: head.forward(x, w, a.double(), i),
        lambda: head.forward(x, w, torch.cat([a, a], 1), torch.cat([i, i], 1)),
        lambda: head.forward(x, w, a.t().contiguous().t(), i),
        lambda: head.forward(x, w, a[:1].expand(20, 5), i),
        lambda: head.forward_backward(x, w, a, i, dx.float(), dw),
        lambda: head.forward_backward(x, w, a, i, dx, dw[:99]),
        lambda: head.forward(x, w, a, i, loss=torch.empty(2, device=DEV)),
        lambda: F.HeadDistill(100, 64, torch.bfloat16, 20, 5, reduction="none"),
        lambda: head.forward(x, w, a, None),
        lambda: F.HeadDistill(100, 64, torch.float64, 20, 5),
    ):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (
        lambda: head.forward_backward(x, w, a, i, x, dw),                       # a gradient over its input
        lambda: head.forward_backward(x, w, a, i, dw[:20], dw),                 # two gradients in one place
        lambda: head.forward(x, w, a, i, token_loss=a.view(-1)[:20]),
        lambda: head.forward_backward(x, w, a, i, dx, dw, grad_scale=float("nan")),
        lambda: F.HeadDistill(100, 64, torch.bfloat16, 20, 0),
        lambda: F.HeadDistill(100, 64, torch.bfloat16, 20, 1025),
        lambda: F.HeadDistill(100, 64, torch.bfloat16, 20, 5, temperature=0.0),
        lambda: F.HeadDistill(100, 64, torch.bfloat16, 20, 5, temperature=float("nan")),
    ):
        with pytest.raises(F.FsdpError):
            bad()
