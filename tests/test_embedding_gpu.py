"""The token embedding and its gradient (fsdp_embed, fsdp_embed_grad, Embedding)
against their definitions in fp64.

Tolerances, derived from the operations (u: half a step of the type, 2^-8 bf16,
2^-11 fp16, 2^-24 fp32, relative to the value; s: half the smallest subnormal
step, 2^-25 of fp16):
* lookup: the factor rounded to fp32, the product rounded to fp32 (2^-24 each,
  2^-23 with their second-order terms) and to the type: u |out| + s.
* gradient: a sum of k fp32 terms in any grouping is within (k - 1) 2^-24 of the
  sum of their magnitudes; the factor, its product and, where it is added, that
  sum 2^-24 each; the type's rounding u |result| + s; second-order terms 1 %.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
STEP = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}
IGNORE = -100


@pytest.fixture(scope="module")
def F():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sharded_fsdp_reduce_gb300 as F
    return F


def tokens_of(kind, T, V, g):
    if kind == "same":
        return torch.full((T,), V // 2, dtype=torch.int64, device=DEV)
    if kind == "skewed":  # the most common one in a tenth of the places
        u = torch.rand(T, device=DEV, dtype=torch.float64, generator=g)
        return (torch.exp(u * math.log(V + 1.0)).long() - 1).clamp_(0, V - 1)
    if kind == "ends":  # the first and the last row, in runs and alone
        t = torch.zeros(T, dtype=torch.int64, device=DEV)
        t[torch.rand(T, device=DEV, generator=g) < 0.5] = V - 1
        return t
    if kind == "none":
        return torch.full((T,), IGNORE, dtype=torch.int64, device=DEV)
    t = torch.randint(0, V, (T,), device=DEV, generator=g)
    if kind == "padded":
        t[T - T // 3:] = IGNORE
    elif kind == "holes":
        t[torch.rand(T, device=DEV, generator=g) < 0.3] = IGNORE
    return t


def inputs(T, V, D, dt, kind="padded", seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    tokens = tokens_of(kind, T, V, g)
    w = (torch.empty(V, D, device=DEV).normal_(generator=g) * 0.1).to(DT[dt])
    dy = (torch.empty(T, D, device=DEV).normal_(generator=g) * 0.1).to(DT[dt])
    return tokens, w, dy


def check_lookup(out, tokens, w, dt, scale=1.0):
    live = tokens != IGNORE
    want = torch.zeros(out.shape, dtype=torch.float64, device=DEV)
    want[live] = w[tokens[live]].double() * scale
    assert bool((out[~live] == 0).all())
    bound = (U[dt] + 2.0 ** -23) * want.abs() * 1.01 + STEP[dt]
    err = (out.double() - want).abs()
    assert bool((err <= bound).all()), f"off by {float((err / bound).max()):.3g} of what is allowed"


def gradient(tokens, dy, V, scale=1.0):
    """The gradient, the sums of magnitudes and the counts, in fp64."""
    live = tokens != IGNORE
    at = tokens[live]
    total = torch.zeros(V, dy.shape[1], dtype=torch.float64, device=DEV)
    size = torch.zeros_like(total)
    total.index_put_((at,), dy[live].double(), accumulate=True)
    size.index_put_((at,), dy[live].double().abs(), accumulate=True)
    return total * scale, size * abs(scale), torch.bincount(at, minlength=V)


def check_gradient(got, tokens, dy, dt, scale=1.0, before=None):
    total, size, count = gradient(tokens, dy, got.shape[0], scale)
    want = total if before is None else before.double() + total
    bound = 1.01 * 2.0 ** -24 * ((count.clamp(min=1) + 2)[:, None] * size + want.abs()) + U[dt] * want.abs() + STEP[dt]
    err = (got.double() - want).abs()
    over = err > bound
    assert not bool(over.any()), (f"{int(over.sum())} of {over.numel()} beyond the bound, first at "
                                  f"{over.nonzero()[0].tolist()}, worst ratio {float((err / bound).max()):.3g}")
    unused = count == 0
    if before is None:
        assert not bool(got[unused].any())
    else:
        assert torch.equal(got[unused], before[unused])


SIZES = [  # tokens, vocab, dim: words of 16 bytes and not, slices of 512 and 1024 columns and their edges
    (1, 1, 1), (1, 1000, 64), (3, 7, 8), (8, 2, 24), (9, 300, 130), (33, 1000, 520), (64, 1003, 1024), (100, 50, 1032),
    (257, 5000, 72), (1000, 70000, 100), (1025, 300, 1283), (2049, 1024, 264), (4100, 1023, 48), (9000, 140000, 16),
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_lookup(F, T, V, D, dt):
    tokens, w, _ = inputs(T, V, D, dt)
    check_lookup(F.Embedding(V, D, DT[dt], T).forward(tokens, w), tokens, w, dt)
    scale = math.sqrt(D)
    out = torch.full((T, D), 3.0, dtype=DT[dt], device=DEV)
    F.Embedding(V, D, DT[dt], T, scale=scale, grad=False).forward(tokens, w, out=out)
    check_lookup(out, tokens, w, dt, scale)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_gradient(F, T, V, D, dt):
    tokens, w, dy = inputs(T, V, D, dt)
    table = F.Embedding(V, D, DT[dt], T, scale=0.37)
    dw = torch.full_like(w, float("nan"))
    assert table.backward(tokens, dy, dw) is dw
    check_gradient(dw, tokens, dy, dt, 0.37)
    dw = w.clone()
    table.backward(tokens, dy, dw, accumulate=True)
    check_gradient(dw, tokens, dy, dt, 0.37, before=w)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["same", "skewed", "ends", "none", "holes", "uniform"])
@pytest.mark.parametrize("T,V,D", [(7, 3, 40), (100, 1000, 64), (1500, 33, 200), (5000, 2000, 1025), (20000, 50257, 72)])
def test_gradient_of_repeated_tokens(F, T, V, D, kind, dt):
    tokens, w, dy = inputs(T, V, D, dt, kind, seed=3)
    for before in (None, w):
        dw = torch.full_like(w, float("nan")) if before is None else before.clone()
        F.fsdp_embed_grad(tokens, dy, dw, accumulate=before is not None)
        check_gradient(dw, tokens, dy, dt, before=before)


@pytest.mark.parametrize("T", [1023, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 131072, 131073, 270001])
@pytest.mark.parametrize("V", [1000, 1 << 17])
def test_tokens_in_order_at_every_size_of_the_sort(F, T, V):
    """Integers of few bits add up exactly in any order; which rows add up shows."""
    g = torch.Generator(device=DEV).manual_seed(T)
    tokens = tokens_of("skewed", T, V, g)
    tokens[torch.rand(T, device=DEV, generator=g) < 0.1] = IGNORE
    dy = torch.randint(-8, 9, (T, 8), device=DEV, generator=g).float()
    dw = torch.full((V, 8), float("nan"), device=DEV)
    F.fsdp_embed_grad(tokens, dy, dw)
    live = tokens != IGNORE
    want = torch.zeros(V, 8, dtype=torch.float64, device=DEV).index_put_((tokens[live],), dy[live].double(),
                                                                        accumulate=True)
    assert torch.equal(dw.double(), want)


def test_a_vocabulary_of_three_digits(F):
    # tokens of 21 bits: three passes of the sort
    V, D, T = (1 << 20) + 5, 8, 3000
    tokens, _, dy = inputs(T, V, D, "bf16", "uniform")
    tokens[:3] = torch.tensor([V - 1, 0, V - 1], device=DEV)
    dw = torch.full((V, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    F.fsdp_embed_grad(tokens, dy, dw)
    check_gradient(dw, tokens, dy, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off,pad", [(0, 8), (8, 24), (1, 0), (3, 5), (4, 4), (2, 6)])
def test_views_at_any_offset_and_stride(F, off, pad, dt):
    T, V, D = 70, 300, 136
    tokens, w0, dy0 = inputs(T, V, D, dt, "holes", seed=6)

    def place(rows, src=None):
        buf = torch.full((off + rows * (D + pad) + 64,), 7.0, dtype=DT[dt], device=DEV)
        v = buf[off:off + rows * (D + pad)].view(rows, D + pad)[:, :D]
        if src is not None:
            v.copy_(src)
        return buf, v

    def others(buf, v, rows):  # nothing beside the result is written
        v.zero_()
        assert int((buf == 7).sum()) == buf.numel() - rows * D

    table = F.Embedding(V, D, DT[dt], T)
    _, w = place(V, w0)
    buf, out = place(T)
    check_lookup(table.forward(tokens, w, out=out), tokens, w0, dt)
    others(buf, out, T)
    _, dy = place(T, dy0)
    for before in (None, w0):
        buf, dw = place(V, before)
        table.backward(tokens, dy, dw, accumulate=before is not None)
        check_gradient(dw, tokens, dy0, dt, before=before)
        others(buf, dw, V)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_no_tokens(F, dt):
    table = F.Embedding(50, 24, DT[dt], 10)
    tokens = torch.empty(0, dtype=torch.int64, device=DEV)
    rows = torch.empty(0, 24, dtype=DT[dt], device=DEV)
    dw = torch.ones(50, 24, dtype=DT[dt], device=DEV)
    assert table.forward(tokens, dw).shape == (0, 24)
    table.backward(tokens, rows, dw, accumulate=True)
    assert bool((dw == 1).all())
    table.backward(tokens, rows, dw)
    assert not bool(dw.any())
    F.fsdp_embed_grad(tokens, rows, dw)


@pytest.mark.parametrize("D", [64, 65])
def test_tokens_outside_the_vocabulary(F, D):
    """Their rows show as NaN; they have no gradient."""
    V, T = 100, 40
    tokens, w, dy = inputs(T, V, D, "bf16", "uniform")
    bad = tokens.clone()
    for k, t in enumerate((V, -1, 2 ** 40, -2 ** 40, 2 ** 32 + 5, -99)):
        bad[3 * k] = t
    bad[1] = IGNORE
    out = F.Embedding(V, D, torch.bfloat16, T).forward(bad, w)
    wrong = ((bad < 0) | (bad >= V)) & (bad != IGNORE)
    assert int(wrong.sum()) == 6 and bool(torch.isnan(out[wrong]).all())
    check_lookup(out[~wrong], bad[~wrong], w, "bf16")
    dy[wrong] = float("nan")
    dw = torch.full_like(w, float("nan"))
    F.fsdp_embed_grad(bad, dy, dw)
    check_gradient(dw, torch.where(wrong, IGNORE, bad), dy, "bf16")


def test_an_ignored_token_of_the_vocabulary(F):
    """ignore_index may be a row of the table, as a padding token's is."""
    V, D, T = 60, 48, 200
    tokens, w, dy = inputs(T, V, D, "f16", "uniform")
    tokens[::3] = 7
    w[7] = float("nan")
    table = F.Embedding(V, D, torch.float16, T, ignore_index=7)
    as_padding = torch.where(tokens == 7, IGNORE, tokens)
    check_lookup(table.forward(tokens, w), as_padding, w, "f16")
    dw = torch.full_like(w, float("nan"))
    table.backward(tokens, dy, dw)
    check_gradient(dw, as_padding, dy, "f16")
    before = torch.ones_like(w)
    dw = before.clone()
    table.backward(tokens, dy, dw, accumulate=True)
    check_gradient(dw, as_padding, dy, "f16", before=before)


@pytest.mark.parametrize("D", [64, 65])
def test_what_lies_in_ignored_rows_does_not_matter(F, D):
    tokens, w, dy = inputs(300, 100, D, "bf16", "holes")
    dy[tokens == IGNORE] = float("nan")
    dw = torch.full_like(w, float("nan"))
    F.fsdp_embed_grad(tokens, dy, dw)
    check_gradient(dw, tokens, dy, "bf16")


def test_values_that_are_not_finite_stay_in_their_row(F):
    V, D, T = 40, 72, 100
    tokens, w, dy = inputs(T, V, D, "bf16", "uniform")
    tokens[tokens == 5] = 6
    tokens[tokens == 9] = 6
    tokens[[10, 50]], tokens[[20, 60]] = 5, 9
    dy[10, 3] = float("inf")
    dy[20, 4], dy[60, 4] = float("inf"), -float("inf")
    dw = torch.empty_like(w)
    F.fsdp_embed_grad(tokens, dy, dw)
    assert float(dw[5, 3]) == float("inf") and math.isnan(float(dw[9, 4]))
    finite = torch.isfinite(dw)
    assert int((~finite).sum()) == 2
    w[5, 1], w[9, 2] = float("nan"), -float("inf")
    out = F.Embedding(V, D, torch.bfloat16, T).forward(tokens, w)
    want = w[tokens]
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out.nan_to_num(), want.nan_to_num())


def test_gradient_against_differences(F):
    """<out(w + h d) - out(w - h d), dy> / 2h = <dw, d>: out is linear in w, so
    the two differ by fp32's roundings alone: of out, 2^-23 of |out| (two
    roundings) on either side over 2h, and of dw's sums."""
    V, D, T = 50, 40, 300
    tokens, w, dy = inputs(T, V, D, "f32", "holes")
    table = F.Embedding(V, D, torch.float32, T, scale=1.7)
    d = torch.empty_like(w).normal_(generator=torch.Generator(device=DEV).manual_seed(2))
    dw = table.backward(tokens, dy, torch.empty_like(w))
    h = 2.0 ** -3
    up, down = (table.forward(tokens, w + s * h * d) for s in (1, -1))
    slope = float(((up.double() - down.double()) * dy.double()).sum()) / (2 * h)
    want = float((dw.double() * d.double()).sum())
    # w + h d is rounded too
    lookup = 3 * 2.0 ** -23 * float(((up.abs() + down.abs()).double() * dy.abs().double()).sum()) / (2 * h)
    _, size, count = gradient(tokens, dy, V, 1.7)
    sums = 2.0 ** -23 * float(((count + 3)[:, None] * size * d.abs().double()).sum())
    assert abs(slope - want) <= lookup + sums, (slope, want)


def test_same_bits_every_time(F):
    tokens, w, dy = inputs(5000, 2000, 264, "bf16", "skewed")
    a = [F.Embedding(2000, 264, torch.bfloat16, 5000).backward(tokens, dy, torch.empty_like(w)) for _ in range(4)]
    assert all(torch.equal(a[0], b) for b in a[1:])


def test_one_table_for_calls_of_many_sizes_and_streams(F):
    V, D, most = 3000, 136, 5000
    table = F.Embedding(V, D, torch.bfloat16, most)
    s = torch.cuda.Stream()
    for k, T in enumerate((most, 1, 37, 1025, 8, 4999)):
        tokens, w, dy = inputs(T, V, D, "bf16", "skewed", seed=k)
        dw = torch.empty_like(w)
        s.wait_stream(torch.cuda.current_stream())
        out = table.forward(tokens, w, stream=s)
        table.backward(tokens, dy, dw, stream=s)
        table.backward(tokens, dy, dw, accumulate=True, stream=s)
        s.synchronize()
        check_lookup(out, tokens, w, "bf16")
        total, size, count = gradient(tokens, dy, V)
        bound = 2 * (2.0 ** -24 * (count + 4)[:, None] * size + 2.0 ** -8 * total.abs()) * 1.02 + 2 * STEP["bf16"]
        assert bool(((dw.double() - 2 * total).abs() <= bound).all())


def test_tokens_of_any_shape(F):
    tokens, w, dy = inputs(60, 100, 64, "bf16", "holes")
    table = F.Embedding(100, 64, torch.bfloat16, 60)
    assert torch.equal(table.forward(tokens.view(4, 15), w), table.forward(tokens, w))


def test_captured_in_a_graph(F):
    T, V, D = 2000, 1200, 128
    tokens, w, dy = inputs(T, V, D, "bf16")
    table = F.Embedding(V, D, torch.bfloat16, T)
    out, dw, tied = torch.empty_like(dy), torch.empty_like(w), torch.empty_like(w)
    for f in (lambda: table.forward(tokens, w, out=out), lambda: table.backward(tokens, dy, dw),
              lambda: table.backward(tokens, dy, tied, accumulate=True)):
        f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        table.forward(tokens, w, out=out)
        table.backward(tokens, dy, dw)
        table.backward(tokens, dy, tied, accumulate=True)
    for k in range(2):
        t2, w2, dy2 = inputs(T, V, D, "bf16", "skewed", seed=30 + k)
        tokens.copy_(t2), w.copy_(w2), dy.copy_(dy2), tied.copy_(w2)
        g.replay()
        torch.cuda.synchronize()
        check_lookup(out, t2, w2, "bf16")
        check_gradient(dw, t2, dy2, "bf16")
        check_gradient(tied, t2, dy2, "bf16", before=w2)


def test_two_graphs_and_eager_calls_share_a_workspace(F):
    T, V, D = 3000, 500, 264
    table = F.Embedding(V, D, torch.bfloat16, T)
    sets = [inputs(T, V, D, "bf16", "skewed", seed=k) for k in range(3)]
    outs = [torch.empty(V, D, dtype=torch.bfloat16, device=DEV) for _ in sets]
    for (tokens, _, dy), dw in zip(sets, outs):
        table.backward(tokens, dy, dw)
    torch.cuda.synchronize()
    graphs = []
    for (tokens, _, dy), dw in zip(sets[:2], outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            table.backward(tokens, dy, dw)
        graphs.append(g)
    for dw in outs:
        dw.fill_(float("nan"))
    graphs[1].replay()
    table.backward(sets[2][0], sets[2][2], outs[2])
    graphs[0].replay()
    torch.cuda.synchronize()
    for (tokens, _, dy), dw in zip(sets, outs):
        check_gradient(dw, tokens, dy, "bf16")


def test_a_workspace_waits_for_its_memorys_last_user(F):
    from sharded_fsdp_reduce_gb300 import embedding as mod
    T, V, D = 60000, 500, 8
    tokens, w, dy = inputs(T, V, D, "bf16", "uniform")
    dw = torch.empty_like(w)
    F.fsdp_embed_grad(tokens, dy, dw)
    need = mod._workspace_bytes(mod._grad_args(tokens, dy, dw, 1.0, IGNORE, False))
    for form in ("function", "object"):
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        block = torch.full((need,), 7, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        copy = block.clone()  # still to be made when the block is back with the allocator
        del block
        if form == "function":
            F.fsdp_embed_grad(tokens, dy, dw, stream=s)
        else:
            F.Embedding(V, D, torch.bfloat16, T).backward(tokens, dy, dw, stream=s)
        torch.cuda.synchronize()
        assert bool((copy == 7).all())
        check_gradient(dw, tokens, dy, "bf16")


def test_tables_longer_than_32_bits_of_elements(F):
    V, D, T = (1 << 18) + 3, 8200, 60  # 2^31 elements and more, rows on both sides of it
    w = torch.zeros(V, D, dtype=torch.bfloat16, device=DEV)
    tokens = torch.randint(V - 40, V, (T,), device=DEV)
    tokens[:4] = torch.tensor([0, 1, V - 1, V - 40], device=DEV)
    w[tokens] = torch.randn(T, D, device=DEV, dtype=torch.bfloat16)
    table = F.Embedding(V, D, torch.bfloat16, T)
    assert torch.equal(table.forward(tokens, w), w[tokens])
    dy = torch.randint(-4, 5, (T, D), device=DEV).to(torch.bfloat16)  # sums of up to 60 of them are exact
    w.fill_(float("nan"))
    table.backward(tokens, dy, w)
    want = torch.zeros(V, D, dtype=torch.bfloat16, device=DEV)
    for k in range(T):
        want[tokens[k]] += dy[k]
    assert torch.equal(w, want)


def test_refusals(F):
    tokens, w, dy = inputs(20, 100, 64, "bf16")
    table = F.Embedding(100, 64, torch.bfloat16, 20)
    dw = torch.empty_like(w)
    for bad in (
        lambda: table.forward(tokens, w.float()),
        lambda: table.forward(tokens, w[:50]),
        lambda: table.forward(torch.cat([tokens, tokens]), w),
        lambda: table.forward(tokens.int(), w),
        lambda: table.forward(tokens.cpu(), w),
        lambda: table.forward(tokens[::2], w),
        lambda: table.forward(tokens, w.cpu()),
        lambda: table.forward(tokens, w, out=dy[:10]),
        lambda: table.forward(tokens, w, out=dy.float()),
        lambda: table.forward(tokens, w, out=dy[:1].expand(20, 64)),
        lambda: table.forward(tokens, w, out=torch.empty(64, 20, dtype=torch.bfloat16, device=DEV).t()),
        lambda: table.backward(tokens, dy[:10], dw),
        lambda: table.backward(tokens, dy.float(), dw),
        lambda: table.backward(tokens, dy, dw[:99]),
        lambda: table.backward(tokens, dy, None),
        lambda: table.backward(tokens, None, dw),
        lambda: F.Embedding(100, 64, torch.bfloat16, 20, grad=False).backward(tokens, dy, dw),
    ):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(TypeError):
        F.Embedding(100, 64, torch.float64, 20)
    both = torch.empty(120, 64, dtype=torch.bfloat16, device=DEV)
    for bad in (
        lambda: table.forward(tokens, w, out=w[:20]),                  # over its input
        lambda: table.backward(tokens, both[90:110], both[:100]),
        lambda: F.Embedding(100, 64, torch.bfloat16, -1),
        lambda: F.Embedding(0, 64, torch.bfloat16, 20),
        lambda: F.Embedding(100, 64, torch.bfloat16, 20, scale=float("nan")),
        lambda: F.fsdp_embed(tokens, w, torch.empty_like(dy), scale=float("inf")),
    ):
        with pytest.raises(F.FsdpError):
            bad()
