"""The global gradient norm, clipping of tensor lists, and the clipped model
step, against fp64 and against the unclipped step's bits.

Tolerance of a norm: eight squares are added in fp32 (each of at most eight
roundings of 2^-24 of the sum), the rest in fp64, the root and the result
rounded once: 2^-21 relative, with room.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NORM_RTOL = 2.0 ** -21


@pytest.fixture(scope="module")
def F():
    import __graft_entry__ as g
    g.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sharded_fsdp_reduce_gb300 as F
    return F


def rand(n, dtype, seed, sigma=1e-2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.empty(n, device=DEV).normal_(generator=g) * sigma).to(dtype)


def norm64(tensors, scale=1.0):
    return abs(scale) * math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


def factor(norm, max_norm, scale=1.0):
    """The factor the definition gives in fp32, one rounding per operation."""
    q = torch.tensor(max_norm, dtype=F32, device=DEV) / (norm + torch.tensor(1e-6, dtype=F32, device=DEV))
    return torch.tensor(scale, dtype=F32, device=DEV) * torch.where(q >= 1, torch.ones_like(q), q)


def assert_norm(got, want):
    assert abs(float(got) - want) <= NORM_RTOL * want, (float(got), want)


LISTS = [
    [1], [7], [8], [9], [2048], [2049, 1, 0, 8191], [0, 0, 5], [3, 100_003, 65_536, 12], [17] * 700, [1_000_003],
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip_in_place(F, sizes, dtype):
    ts = [rand(n, dtype, 10 + i) for i, n in enumerate(sizes)]
    want = norm64(ts)
    ref = [t.clone() for t in ts]
    clip = F.GradClip(ts)
    norm = clip.norm().clone()
    assert_norm(norm, want)
    assert torch.equal(clip.norm(), norm)  # the workspace is ready again, the order fixed
    got = clip.clip(0.25 * want)
    assert torch.equal(got, norm)
    f = factor(norm, 0.25 * want)
    for t, r in zip(ts, ref):
        assert torch.equal(t, (r.float() * f).to(dtype))


def test_mixed_dtypes_and_unaligned_views(F):
    flat = [rand(50_000, dt, 3) for dt in (F32, BF16, F16)]
    outs = [torch.full((50_000,), float("nan"), dtype=f.dtype, device=DEV) for f in flat]
    ts, os_ = [], []
    for k, (f, o) in enumerate(zip(flat, outs)):
        for lo, n, at in ((1, 999, 3), (1003, 8, 1005), (2001, 30_011, 2001), (40_000, 1, 40_007), (40_001, 4097, 41_004)):
            ts.append(f[lo:lo + n])
            os_.append(o[at:at + n])
    clip = F.GradClip(ts, out=os_, scale=0.5)
    norm = clip.clip(0.01)
    assert_norm(norm, norm64(ts, 0.5))
    f = factor(norm, 0.01, 0.5)
    written = [torch.zeros(50_000, dtype=torch.bool, device=DEV) for _ in flat]
    for i, (t, o) in enumerate(zip(ts, os_)):
        assert torch.equal(o, (t.float() * f).to(t.dtype)), i
        k = i // 5
        lo = (o.data_ptr() - outs[k].data_ptr()) // o.element_size()
        written[k][lo:lo + o.numel()] = True
    for o, w in zip(outs, written):  # nothing beside them is touched
        assert bool(torch.isnan(o[~w].float()).all())


def test_no_clipping_below_the_limit_leaves_the_bits(F):
    t = rand(12_345, BF16, 1)
    ref = t.clone()
    out = torch.zeros_like(t)
    F.GradClip([t]).clip(1e3)
    assert torch.equal(t, ref)
    F.GradClip([t], out=[out]).clip(float("inf"))
    assert torch.equal(out, ref)


@pytest.mark.parametrize("value", [1e30, 3e37, 1e-25, 1e-38, 1e-42])
def test_norm_where_squares_leave_fp32(F, value):
    t = torch.full((10_007,), value, dtype=F32, device=DEV)
    t[5000:] = 0
    want = norm64([t])
    got = float(F.GradClip([t]).norm())
    if want > 3.4e38:
        assert math.isinf(got)
    else:
        assert abs(got - want) <= NORM_RTOL * want + 2.0 ** -149


def test_norm_mixes_small_and_large(F):
    t = rand(4096, F32, 2)
    t[7] = 2e25
    t[2000] = 1e-30
    assert_norm(F.GradClip([t]).norm(), norm64([t]))


@pytest.mark.parametrize("bad,want", [(float("nan"), "nan"), (float("inf"), "inf"), (float("-inf"), "inf")])
def test_norm_of_values_that_are_not_finite(F, bad, want):
    t = rand(30_000, F32, 4)
    t[12_345] = bad
    clip = F.GradClip([t])
    n = float(clip.norm())
    assert math.isnan(n) if want == "nan" else math.isinf(n)
    clip.clip(1.0)
    if want == "nan":
        assert bool(torch.isnan(t).all())
    else:
        assert math.isnan(float(t[12_345])) and not bool(t[:12_345].any()) and not bool(t[12_346:].any())


def test_all_zero_and_empty(F):
    z = torch.zeros(5000, device=DEV)
    assert float(F.GradClip([z]).clip(1.0)) == 0.0 and not bool(z.any())
    e = torch.empty(0, device=DEV)
    assert float(F.GradClip([e, e]).clip(1.0)) == 0.0
    assert float(F.GradClip([]).clip(1.0)) == 0.0


def test_elements_past_32_bits(F):
    n = 2 ** 31 + 4099
    t = torch.zeros(n, dtype=BF16, device=DEV)
    t[-1], t[2 ** 31], t[0] = 3.0, 4.0, 12.0
    clip = F.GradClip([t])
    assert float(clip.clip(6.5)) == 13.0
    f = float(factor(torch.tensor(13.0, device=DEV), 6.5))
    for at, v in ((n - 1, 3.0), (2 ** 31, 4.0), (0, 12.0)):
        assert float(t[at]) == float(torch.tensor(v * f).to(BF16))


def test_on_another_stream_than_it_was_made_on(F):
    s = torch.cuda.Stream()
    for k in range(5):
        t = rand(300_000 + k, F32, k)
        clip = F.GradClip([t])
        s.wait_stream(torch.cuda.current_stream())
        norm = clip.norm(torch.empty((), device=DEV), stream=s)
        del clip
        torch.zeros(10_000, dtype=torch.uint8, device=DEV).fill_(255)  # would land in the freed workspace
        s.synchronize()
        assert_norm(norm, norm64([t]))


def test_its_own_norm_on_another_stream_while_the_first_is_busy(F, monkeypatch):
    """Whatever the object prepares on the stream it was made on is done
    before a call on another stream: every fill is made to come late here."""
    s = torch.cuda.Stream()
    t = rand(100_003, F32, 1)
    ref, want = t.clone(), norm64([t])
    F.GradClip([t.clone()]).clip(1.0)  # (a kernel's first launch waits for the device)
    zeros = torch.zeros

    def late(*args, **kw):
        torch.cuda._sleep(20_000_000)
        return zeros(*args, **kw)

    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "zeros", late)
    clip = F.GradClip([t])
    monkeypatch.undo()
    norm = clip.clip(0.25 * want, stream=s)
    torch.cuda.synchronize()
    assert_norm(norm, want)
    assert torch.equal(t, ref * factor(norm, 0.25 * want))


def test_its_own_norm_is_held_for_the_stream(F):
    s = torch.cuda.Stream()
    t = rand(100_003, F32, 1)
    clip = F.GradClip([t])
    clip.clip(1.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)
    clip.clip(0.1, stream=s)
    del clip
    others = [torch.full((), 7.0, device=DEV) for _ in range(4000)]  # would land in freed blocks of its size
    torch.cuda.synchronize()
    assert all(float(x) == 7.0 for x in others)


def test_captured_in_a_graph(F):
    t = rand(70_001, BF16, 9)
    out = torch.empty_like(t)
    clip = F.GradClip([t], out=[out])
    norm = torch.empty((), device=DEV)
    clip.norm(norm)
    clip.clip(1.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        clip.norm(norm)
        clip.clip(0.5, norm)
    for k in range(3):
        t.copy_(rand(70_001, BF16, 20 + k))
        g.replay()
        torch.cuda.synchronize()
        assert_norm(norm, norm64([t]))
        assert torch.equal(out, (t.float() * factor(norm, 0.5)).to(BF16))


def test_made_within_a_capture_and_used_outside_it(F):
    t = rand(70_001, F32, 9)
    u = make_units(F, [9001], 8, BF16, BF16, 15, n_full=1)
    F.GradClip([t.clone()]).clip(1.0)
    F.UnitSequence(make_units(F, [9001], 8, BF16, BF16, 15, n_full=1)).clip_step(F.AdamWHParams(**HP), 0.05)
    want, step_want = norm64([t]), norm64([average(u[0], 1.0)])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        junk = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)
        del junk  # (what the graph's memory holds is not 0)
        clip, model = F.GradClip([t]), F.UnitSequence(u)
        norm = clip.norm(torch.empty((), device=DEV))
        step_norm = model.clip_step(F.AdamWHParams(**HP), 0.05)
    assert_norm(clip.norm(), want)
    assert_norm(model.clip_step(F.AdamWHParams(**HP), 0.05), step_want)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert_norm(norm, want)
        assert_norm(step_norm, step_want)
    assert_norm(clip.norm(), want)


def test_refusals(F):
    t = rand(100, F32, 0)
    with pytest.raises(ValueError):
        F.GradClip([t.cpu()])
    with pytest.raises(ValueError):
        F.GradClip([t.reshape(10, 10).t()])
    with pytest.raises(TypeError):
        F.GradClip([t.double()])
    with pytest.raises(ValueError):
        F.GradClip([t], out=[t[:50]])
    with pytest.raises(ValueError):
        F.GradClip([t], out=[torch.empty(100, dtype=BF16, device=DEV)])
    clip = F.GradClip([t])
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(F.FsdpError):
            clip.clip(bad)
    with pytest.raises(F.FsdpError):  # two results in one place
        F.GradClip([t[:50], t[50:]], out=[t[:50], t[:50]]).clip(1.0)
    with pytest.raises(F.FsdpError):  # a result over another's source
        F.GradClip([t[:50], t[50:]], out=[t[50:], t[:50]]).clip(1.0)
    with pytest.raises(F.FsdpError):  # shifted over itself
        F.GradClip([t[:50]], out=[t[1:51]]).clip(1.0)
    with pytest.raises(ValueError):
        clip.norm(torch.empty(2, device=DEV))


# ---------------------------------------------------------------- the clipped step


def make_units(F, sizes, world, gdt, odt, seed, n_full=None, scale=1.0, **kw):
    units = []
    for k, n in enumerate(sizes):
        u = F.FlatParamUnit([("w", (n,))], world, gdt, odt, device=DEV, n_full=n_full, **kw)
        u.load_master([rand(n, F32, seed + 100 * k, 0.1)])
        u.exp_avg[:n] = rand(n, F32, seed + 100 * k + 1, 1e-3).to(u.exp_avg.device)
        u.exp_avg_sq[:n] = rand(n, F32, seed + 100 * k + 2, 1e-3).square().to(u.exp_avg.device)
        for r in range(world):
            u.load_grad(r, [rand(n, F32, seed + 100 * k + 3 + r, 1e-2 * scale).to(gdt)])
        units.append(u)
    return units


def average(u, scale):
    acc = u.grads[0].to(DEV).float()
    for g in u.grads[1:]:
        acc = acc + g.to(DEV).float()
    return acc * torch.tensor(1.0 / (u.world * scale), dtype=F32, device=DEV)


def check_step(F, make, hp, share, gathers=1, stream=None, **kw):
    """clip_step against the fused kernel run on the clipped average as one rank's fp32 gradient."""
    a, b = make(), make()
    avg = [average(u, hp.grad_scale) for u in a]
    want = norm64(avg)
    norm = F.UnitSequence(a).clip_step(hp, share * want, gathers=gathers, stream=stream, **kw)
    torch.cuda.synchronize()
    assert_norm(norm, want)
    coef = factor(norm, share * want)
    one = F.AdamWHParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, hp.step, 1.0)
    for ua, ub, g in zip(a, b, avg):
        if not g.numel():
            continue
        F.fsdp_reduce_scatter_adam_cast([g * coef], ub.master, ub.exp_avg, ub.exp_avg_sq, ub.shard_out, one)
        torch.cuda.synchronize()
        for name in ("master", "exp_avg", "exp_avg_sq"):
            assert torch.equal(getattr(ua, name).view(torch.int32), getattr(ub, name).view(torch.int32)), name
        assert torch.equal(ua.shard_out, ub.shard_out)
        for f in ua.full if gathers else []:
            assert torch.equal(f, ub.shard_out)


HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=7)


@pytest.mark.parametrize("world", [1, 2, 3, 4, 5, 8, 16])
@pytest.mark.parametrize("gdt,odt", [(BF16, BF16), (F16, F16), (F32, BF16), (F32, F32), (BF16, F32)],
                         ids=lambda d: str(d).split(".")[-1])
def test_clipped_step(F, world, gdt, odt):
    scale = 1024.0 if gdt == F16 else 1.0
    make = lambda: make_units(F, [4099, 37, 20_000], world, gdt, odt, 5, n_full=2, scale=scale)  # noqa: E731
    check_step(F, make, F.AdamWHParams(grad_scale=scale, **HP), 0.3)


@pytest.mark.parametrize("gathers,n_full", [(0, 0), (1, 1), (2, 8), (1, 9), (2, 11)])
def test_clipped_step_gathers(F, gathers, n_full):
    make = lambda: make_units(F, [5000, 1, 8200], 8, BF16, BF16, 6, n_full=n_full)  # noqa: E731
    check_step(F, make, F.AdamWHParams(**HP), 0.5, gathers=gathers)


@pytest.mark.parametrize("world,gdt", [(8, BF16), (2, BF16), (2, F32), (4, F16)])
def test_without_clipping_it_is_the_step(F, world, gdt):
    sizes = [4099, 2048, 3, 100_000]
    a = make_units(F, sizes, world, gdt, BF16, 7)
    b = make_units(F, sizes, world, gdt, BF16, 7)
    hp = F.AdamWHParams(**HP)
    F.UnitSequence(a).clip_step(hp, float("inf"))
    F.UnitSequence(b).step(hp)
    torch.cuda.synchronize()
    for ua, ub in zip(a, b):
        for name in ("master", "exp_avg", "exp_avg_sq"):
            assert torch.equal(getattr(ua, name).view(torch.int32), getattr(ub, name).view(torch.int32))
        for fa, fb in zip(ua.full, ub.full):
            assert torch.equal(fa, fb)


def test_clipped_step_many_units(F):
    make = lambda: make_units(F, [11 + 13 * k for k in range(400)], 8, BF16, BF16, 8, n_full=1)  # noqa: E731
    check_step(F, make, F.AdamWHParams(**HP), 0.7)


def test_clipped_step_mixed_model(F):
    def make():
        return (make_units(F, [3000, 0, 17], 8, BF16, BF16, 9) + make_units(F, [999], 3, F32, F16, 10)
                + make_units(F, [40_001], 2, F16, F16, 11) + make_units(F, [6000], 1, F32, F32, 12))
    check_step(F, make, F.AdamWHParams(**HP), 0.4)


def test_clipped_step_offloaded(F):
    make = lambda: make_units(F, [5003, 300], 2, BF16, BF16, 13, state_on_host=True)  # noqa: E731
    check_step(F, make, F.AdamWHParams(**HP), 0.4)


def test_clipped_step_unaligned(F):
    def make():
        units = make_units(F, [4100], 4, BF16, BF16, 14, n_full=1)
        u = units[0]
        for name in ("master", "exp_avg", "exp_avg_sq", "shard_out"):
            t = getattr(u, name)
            buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)
            buf[1:] = t
            setattr(u, name, buf[1:])
        grads = []
        for g in u.grads:
            buf = torch.zeros(g.numel() + 3, dtype=g.dtype, device=DEV)
            buf[3:] = g
            grads.append(buf[3:])
        u.grads = grads
        return units
    check_step(F, make, F.AdamWHParams(**HP), 0.4)


def test_clipped_step_on_another_stream_and_repeated(F):
    s = torch.cuda.Stream()
    units = make_units(F, [9001, 512], 8, BF16, BF16, 15, n_full=1)
    twin = make_units(F, [9001, 512], 8, BF16, BF16, 15, n_full=1)
    model, other = F.UnitSequence(units), F.UnitSequence(twin)
    s.wait_stream(torch.cuda.current_stream())
    for t in range(3):
        hp = F.AdamWHParams(**dict(HP, step=t + 1))
        n1 = model.clip_step(hp, 0.05, stream=s)
        n2 = other.clip_step(hp, 0.05)
        torch.cuda.synchronize()
        assert torch.equal(n1, n2)
    for a, b in zip(units, twin):
        assert torch.equal(a.master, b.master) and torch.equal(a.full[0], b.full[0])


@pytest.mark.parametrize("world,gdt", [(8, BF16), (2, BF16), (1, F32)])
def test_many_clipped_steps_in_a_row(F, world, gdt):
    """Steps that start while the one before drains, on units that fill the
    part: every step reads the state that the one before has written."""
    sizes = [3_000_007, 700_003, 1_000_000, 5]
    a = make_units(F, sizes, world, gdt, BF16, 20, n_full=1)
    b = make_units(F, sizes, world, gdt, BF16, 20, n_full=1)
    clipped, plain = F.UnitSequence(a), F.UnitSequence(b)
    clipped.clip_step(F.AdamWHParams(**dict(HP, step=1)), float("inf"))
    plain.step(F.AdamWHParams(**dict(HP, step=1)))
    torch.cuda.synchronize()
    norm = torch.empty((), device=DEV)
    for t in range(2, 60):
        clipped.clip_step(F.AdamWHParams(**dict(HP, step=t)), float("inf"), norm=norm)
    for t in range(2, 60):
        plain.step(F.AdamWHParams(**dict(HP, step=t)))
    torch.cuda.synchronize()
    for ua, ub in zip(a, b):
        for name in ("master", "exp_avg", "exp_avg_sq"):
            assert torch.equal(getattr(ua, name).view(torch.int32), getattr(ub, name).view(torch.int32)), name
        assert torch.equal(ua.full[0], ub.full[0])
    assert_norm(norm, norm64([average(u, 1.0) for u in a]))


def test_many_clips_in_a_row(F):
    ts = [rand(n, BF16, 40 + n % 7) for n in (2_000_003, 17, 900_001)]
    ref = [t.clone() for t in ts]
    clip = F.GradClip(ts, scale=0.75)
    norms = torch.empty(30, device=DEV)
    for k in range(30):
        clip.norm(norms[k])
        clip.clip(float("inf"), norms[k])
    torch.cuda.synchronize()
    for k in range(30):
        assert_norm(norms[k], norm64(ref, 0.75))
        ref = [(r.float() * 0.75).to(BF16) for r in ref]
    assert all(torch.equal(t, r) for t, r in zip(ts, ref))


def test_a_captured_clipped_step_outlives_a_change_of_arguments(F):
    """A captured graph of clipped steps keeps writing to the workspace that
    they were captured with, whatever plan later calls make."""
    units = make_units(F, [200_003, 512], 8, BF16, BF16, 18, n_full=1)
    twin = make_units(F, [200_003, 512], 8, BF16, BF16, 18, n_full=1)
    model, hp = F.UnitSequence(units), F.AdamWHParams(**HP)
    norm = torch.empty((), device=DEV)
    model.clip_step(hp, 0.05, norm=norm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        model.clip_step(hp, 0.05, norm=norm)
    nf = torch.zeros(1, dtype=torch.int32, device=DEV)
    model.clip_step(hp, 0.05, nonfinite_count=nf)
    model.clip_step(hp, 0.05, gathers=0)
    torch.cuda.synchronize()
    size = model._clip_plan.workspace.buf.numel()
    assert size > 4 * 200_003
    others = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(3)]
    g.replay()
    torch.cuda.synchronize()
    assert all(bool((o == 7).all()) for o in others)
    other = F.UnitSequence(twin)
    for _ in range(4):
        n = other.clip_step(hp, 0.05)
    torch.cuda.synchronize()
    assert torch.equal(n, norm)
    for a, b in zip(units, twin):
        assert torch.equal(a.master, b.master) and torch.equal(a.full[0], b.full[0])


def test_a_larger_plan_keeps_the_earlier_workspace(F):
    # two ranks in 16 bits keep no average; the variant form keeps every one
    model = F.UnitSequence(make_units(F, [50_003], 2, BF16, BF16, 19, n_full=1))
    model.clip_step(F.AdamWHParams(**HP), 0.05)
    first = model._clip_plan.workspace
    model.clip_step(F.StepConfig("adamw", 1e-3, 0.9, 0.95, 1e-8, 0.1, 7), 0.05)
    second = model._clip_plan.workspace
    assert second is not first and any(k is first for k in model._clip_kept)
    model.clip_step(F.AdamWHParams(**HP), 0.05)  # and the smaller plan works in the larger one's
    assert model._clip_plan.workspace is second
    torch.cuda.synchronize()


def test_clipped_step_counts_and_shows_values_that_are_not_finite(F):
    units = make_units(F, [4099, 700], 8, BF16, BF16, 16, n_full=1)
    units[0].grads[3][100] = float("inf")
    units[1].grads[0][5] = float("nan")
    nf = torch.zeros(1, dtype=torch.int32, device=DEV)
    norm = F.UnitSequence(units).clip_step(F.AdamWHParams(**HP), 1.0, nonfinite_count=nf)
    torch.cuda.synchronize()
    assert int(nf) == 2 and math.isnan(float(norm))


def test_clipped_step_refusals(F):
    units = make_units(F, [100], 2, BF16, BF16, 17)
    model = F.UnitSequence(units)
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(F.FsdpError):
            model.clip_step(F.AdamWHParams(**HP), bad)
    with pytest.raises(F.FsdpError):
        model.clip_step(F.AdamWHParams(**dict(HP, step=0)), 1.0)
    sgd = F.FlatParamUnit([("w", (8,))], 2, BF16, BF16, device=DEV, optimizer="sgd")
    with pytest.raises(ValueError):  # an SGD unit steps with a StepConfig
        F.UnitSequence([sgd]).clip_step(F.AdamWHParams(**HP), 1.0)
    with pytest.raises(F.FsdpError):  # the norm is of the fp32 average
        F.UnitSequence([sgd]).clip_step(F.StepConfig("sgd", 1e-3, reduce_dtype=BF16), 1.0)
    with pytest.raises(F.FsdpError):
        F.UnitSequence([sgd]).clip_step(F.StepConfig("sgd", 1e-3), -1.0)
    with pytest.raises(ValueError):
        model.clip_step(F.AdamWHParams(**HP), 1.0, norm=torch.empty(2, device=DEV))


VARIANTS = [("sgd", F32), ("adamax", F32), ("adadelta", F32), ("adamw", BF16), ("sgd", BF16), ("adamax", F16)]


@pytest.mark.parametrize("world", [1, 3, 8])
@pytest.mark.parametrize("optimizer,state", VARIANTS, ids=lambda v: str(v).split(".")[-1])
@pytest.mark.parametrize("share", [0.3, float("inf")])
def test_clipped_variant_step(F, optimizer, state, world, share):
    """Against the variant kernel run on the clipped average as one rank's fp32 gradient."""
    odt = BF16 if state == F32 else state
    scale = 64.0
    make = lambda: make_units(F, [4099, 0, 37, 20_000], world, odt, odt, 21, n_full=2, scale=scale,  # noqa: E731
                              optimizer=optimizer, state_dtype=state) if optimizer != "sgd" else \
        sgd_units(F, [4099, 0, 37, 20_000], world, odt, odt, scale, state)
    a, b = make(), make()
    if optimizer == "adadelta":
        for u in a + b:
            u.exp_avg.abs_()  # its first state is a running mean of squares
    avg = [average(u, scale) for u in a]
    want = norm64(avg)
    cfg = F.StepConfig(optimizer, 1e-3, 0.9, 0.95, 1e-8, 0.1, 7, scale)
    nf = torch.zeros(1, dtype=torch.int32, device=DEV)
    norm = F.UnitSequence(a).clip_step(cfg, share * want, nonfinite_count=nf)
    torch.cuda.synchronize()
    assert_norm(norm, want)
    assert int(nf) == 0
    coef = factor(norm, share * want)
    one = F.StepConfig(optimizer, 1e-3, 0.9, 0.95, 1e-8, 0.1, 7, 1.0)
    for ua, ub, g in zip(a, b, avg):
        if not g.numel():
            continue
        F.fsdp_reduce_scatter_step([g * coef], ub.master, ub.exp_avg, ub.exp_avg_sq,
                                   None if state != F32 else ub.shard_out, one)
        torch.cuda.synchronize()
        for name in ("master", "exp_avg", "exp_avg_sq"):
            x, y = getattr(ua, name), getattr(ub, name)
            assert (x is None and y is None) or torch.equal(x, y), name
        for f in ua.full:
            assert torch.equal(f, ub.shard_out)


def sgd_units(F, sizes, world, gdt, odt, scale, state):
    units = []
    for k, n in enumerate(sizes):
        u = F.FlatParamUnit([("w", (n,))], world, gdt, odt, device=DEV, n_full=2, optimizer="sgd", state_dtype=state)
        u.load_master([rand(n, F32, 50 + k, 0.1)])
        u.exp_avg[:n] = rand(n, F32, 60 + k, 1e-3)
        for r in range(world):
            u.load_grad(r, [rand(n, F32, 70 + 10 * k + r, 1e-2 * scale).to(gdt)])
        units.append(u)
    return units
