"""The distillation loss where its kernels change form: calls of more rows than
eight for each SM, the largest numbers of entries, the temperatures' limits, and
objects that serve calls on both sides of a change. Bounds as in
test_distill_gpu.py."""
import pytest
import torch

from test_distill_gpu import DEV, F, check, inputs, reference, run  # noqa: F401 (F: a fixture)

pytestmark = pytest.mark.gpu


def eight_rows():
    """The longest call whose row kernel has eight rows a block."""
    return 8 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("more", [0, 1, 1284])
@pytest.mark.parametrize("V,D,K", [(301, 72, 9), (1003, 64, 70)])
def test_calls_around_eight_rows_for_each_sm(F, V, D, K, more, dt):
    T = eight_rows() + more
    x, w, a, i = inputs(T, V, D, K, dt, seed=more)
    ref = reference(x, w, a, i, 2.0)
    loss, tok, _, _ = run(F, x, w, a, i, grad=False, tau=2.0)
    check(ref, dt, (V, T), loss, tok)
    loss, tok, dx, dw = run(F, x, w, a, i, tau=2.0)
    check(ref, dt, (V, T), loss, tok, dx, dw)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("more,band", [(0, 512), (1, 512), (700, 300)])
def test_bands_of_long_calls(F, more, band, dt):
    T, V, D, K = eight_rows() + more, 500, 136, 20
    x, w, a, i = inputs(T, V, D, K, dt, seed=4)
    ref = reference(x, w, a, i)
    loss, tok, dx, dw = run(F, x, w, a, i, band=band)
    check(ref, dt, (V, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, x, w, a, i, grad=False, band=band)
    check(ref, dt, (V, T), loss, tok)


@pytest.mark.parametrize("band", [0, 100])
def test_one_head_for_calls_on_both_sides_of_a_change(F, band):
    """Calls of eight rows a block leave twice as many sums as longer ones of
    nearly the same length; the object's workspace has room for both."""
    V, D, K, eight = 700, 64, 40, eight_rows()
    head = F.HeadDistill(V, D, torch.bfloat16, eight + 900, K, band=band)
    at, size = head._ws_at, head._ws_bytes
    for n, (T, k) in enumerate(((eight + 900, K), (eight, K), (eight + 1, 3), (eight - 1, K), (7, K), (eight + 900, 1))):
        x, w, a, i = inputs(T, V, D, k, "bf16", seed=n)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        loss, tok = head.forward_backward(x, w, a, i, dx, dw)
        l2, t2 = head.forward(x, w, a, i)
        ref = reference(x, w, a, i)
        check(ref, "bf16", (V, T), loss, tok, dx, dw)
        check(ref, "bf16", (V, T), l2, t2)
        assert (head._ws_at, head._ws_bytes) == (at, size)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("K", [256, 257, 512, 513, 1023, 1024])
def test_many_entries(F, K, T, dt):
    V, D = 2100, 64
    for kind in ("some", "twice"):
        x, w, a, i = inputs(T, V, D, K, dt, seed=K, kind=kind)
        ref = reference(x, w, a, i)
        loss, tok, dx, dw = run(F, x, w, a, i)
        check(ref, dt, (V, T), loss, tok, dx, dw)
        loss, tok, _, _ = run(F, x, w, a, i, grad=False)
        check(ref, dt, (V, T), loss, tok)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("tau,std,spread", [(1e-3, 0.01, 2e-3), (1e-3, 0.05, 2.0), (1e3, 0.05, 4.0), (1e3, 2.0, 4e3)])
def test_the_temperatures_limits(F, T, tau, std, spread, dt):
    """Logits over the temperature a few apart, thousands apart, and next to
    equal. D is small where the temperature is: a logit's rounding over it stays
    small enough that its square does not count."""
    x, w, a, i = inputs(T, 1500, 16 if tau < 1 else 96, 40, dt, seed=2, std=std, spread=spread)
    ref = reference(x, w, a, i, tau, grad_scale=1.0 / tau)
    loss, tok, dx, dw = run(F, x, w, a, i, tau=tau, grad_scale=1.0 / tau)
    check(ref, dt, (1500, T), loss, tok, dx, dw)
    loss, tok, _, _ = run(F, x, w, a, i, tau=tau, grad=False)
    check(reference(x, w, a, i, tau), dt, (1500, T), loss, tok)


@pytest.mark.parametrize("T", [4, 1300])
def test_two_heads_at_once_on_two_streams(F, T):
    V, D, K = 900, 128, 30
    sets = [inputs(T, V, D, K, "bf16", seed=k) for k in range(2)]
    heads = [F.HeadDistill(V, D, torch.bfloat16, T, K) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[(torch.empty_like(x), torch.empty_like(w)) for _ in range(4)] for x, w, _, _ in sets]
    results = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for k in range(4):
        for n, ((x, w, a, i), head, s) in enumerate(zip(sets, heads, streams)):
            results[n].append(head.forward_backward(x, w, a, i, *outs[n][k], stream=s))
    torch.cuda.synchronize()
    for (x, w, a, i), out, got in zip(sets, outs, results):
        check(reference(x, w, a, i), "bf16", (V, T), *got[0], *out[0])
        for o, g in zip(out[1:], got[1:]):
            assert all(torch.equal(p, q) for p, q in zip((*o, *g), (*out[0], *got[0])))
