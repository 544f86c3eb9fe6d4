"""Host-side checks of the head loss and clipping entry points: workspace sizes
and refusals, with no GPU and nothing enqueued (the addresses are made up and
never read)."""
import ctypes

import pytest

BASE = 1 << 44  # a made-up device address, 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from sharded_fsdp_reduce_gb300 import _lib
    return _lib.load()


@pytest.fixture(scope="module")
def L():
    from sharded_fsdp_reduce_gb300 import _lib
    return _lib


def loss_args(L, T=100, V=1000, D=64, dtype=None, grad=True, **kw):
    a = L.FsdpHeadLossArgs()
    a.dtype = L.FSDP_BF16 if dtype is None else dtype
    a.tokens, a.vocab, a.dim = T, V, D
    step = 1 << 40
    a.hidden, a.weight, a.targets, a.loss, a.token_loss = (BASE + k * step for k in range(5))
    if grad:
        a.d_hidden, a.d_weight = BASE + 5 * step, BASE + 6 * step
    a.ld_hidden = a.ld_weight = a.ld_d_hidden = a.ld_d_weight = D
    a.ignore_index, a.grad_scale = -100, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def workspace(lib, a):
    n = ctypes.c_int64(-1)
    st = lib.fsdp_head_loss_workspace(ctypes.byref(a), ctypes.byref(n))
    return st, n.value


def test_head_loss_workspace(lib, L):
    ok = lambda a: (lambda r: (r[0] == L.FSDP_OK and r[1] > 0, r[1]))(workspace(lib, a))  # noqa: E731
    good, grad = ok(loss_args(L, T=1000, V=50257, D=768))
    assert good and grad >= 2 * 1000 * 50257  # the 16-bit exponentials of one band
    good, losses = ok(loss_args(L, T=1000, V=50257, D=768, grad=False))
    assert good and losses < grad // 5
    good, few = ok(loss_args(L, T=4, V=50257, D=768, grad=False))
    assert good and few < losses
    # packed when TMA cannot address the weight
    good, packed = ok(loss_args(L, T=1000, V=50257, D=768, weight=BASE + (1 << 40) + 2))
    assert good and packed >= grad + 2 * 50257 * 768
    # bands bound the exponentials whatever the tokens: 4 GiB of them, and one
    # fp32 weight gradient
    good, long = ok(loss_args(L, T=1_000_000, V=128_000, D=64))
    assert good and long < (4 << 30) * 1.3 + 4 * 128_000 * 64 + 32 * 1_000_000
    good, small = ok(loss_args(L, T=1_000_000, V=128_000, D=64, band=256))
    assert good and small < long / 5
    st, n = workspace(lib, loss_args(L, T=0))
    assert st == L.FSDP_OK and n == 0


@pytest.mark.parametrize("T,V,D,dtype,band", [
    (2048, 32000, 4096, "bf16", 0), (4096, 128256, 8192, "bf16", 0), (3000, 1003, 200, "f16", 0),
    (700, 5003, 768, "f32", 0), (30, 33, 8, "f32", 0), (9, 40, 72, "bf16", 0), (900, 700, 64, "bf16", 100),
    (70_000, 131_072, 64, "bf16", 0),  # longer than one band's budget: two of about half its length
])
@pytest.mark.parametrize("grads", ["both", "none"])
def test_head_loss_workspace_is_enough_for_every_shorter_call(lib, L, T, V, D, dtype, band, grads):
    """What the longest call needs is enough for all shorter ones, with both
    gradients or one: they may cut a product into more pieces than it does,
    work in one band where it takes two, or run as a few rows."""
    code = dict(f32=L.FSDP_F32, bf16=L.FSDP_BF16, f16=L.FSDP_F16)[dtype]
    for weight in (2 << 40, (2 << 40) + 4):  # aligned, and to be packed
        kw = dict(V=V, D=D, dtype=code, band=band, weight=BASE + weight, grad=grads != "none")
        st, most = workspace(lib, loss_args(L, T=T, **kw))
        assert st == L.FSDP_OK
        for t in list(range(1, 600)) + list(range(600, T, max(1, T // 3000))):
            if t >= T:
                break
            for alone in (dict(), dict(d_hidden=None), dict(d_weight=None)) if kw["grad"] else (dict(),):
                st, n = workspace(lib, loss_args(L, T=t, **kw, **alone))
                assert st == L.FSDP_OK and n <= most, (t, alone, n, most)


def test_head_loss_refuses(lib, L):
    bad = L.FSDP_ERR_INVALID_ARG
    cases = [
        (dict(dtype=7), L.FSDP_ERR_UNSUPPORTED_DTYPE),
        (dict(tokens=-1), bad), (dict(vocab=0), bad), (dict(dim=0), bad), (dict(tokens=1 << 40), bad),
        (dict(band=-1), bad), (dict(reduction=2), bad), (dict(reserved=1), bad),
        (dict(grad_scale=float("inf")), bad), (dict(grad_scale=float("nan")), bad),
        (dict(hidden=None), bad), (dict(weight=None), bad), (dict(targets=None), bad), (dict(loss=None), bad),
        (dict(ld_hidden=63), bad), (dict(ld_weight=0), bad), (dict(ld_d_weight=-64), bad),
        (dict(ld_hidden=1 << 50), bad),
        (dict(hidden=BASE + 1), L.FSDP_ERR_ALIGNMENT), (dict(targets=BASE + 4), L.FSDP_ERR_ALIGNMENT),
        (dict(loss=BASE + 2), L.FSDP_ERR_ALIGNMENT), (dict(wait_timeouts=BASE + 2), L.FSDP_ERR_ALIGNMENT),
        (dict(d_hidden=BASE), bad),                        # over hidden
        (dict(d_weight=BASE + (1 << 40) + 128), bad),      # into the weight
        (dict(d_hidden=BASE + 6 * (1 << 40)), bad),        # over the other gradient
        (dict(loss=BASE + 4 * (1 << 40)), bad),            # a token's loss
    ]
    for kw, want in cases:
        st, _ = workspace(lib, loss_args(L, **kw))
        assert st == want, kw
        st = lib.fsdp_head_loss(ctypes.byref(loss_args(L, **kw)), BASE + 8 * (1 << 40), 1 << 40, None)
        assert st == want, kw
    assert lib.fsdp_head_loss(None, BASE, 1 << 40, None) == bad
    assert lib.fsdp_head_loss_workspace(ctypes.byref(loss_args(L)), None) == bad
    a = loss_args(L)
    _, need = workspace(lib, a)
    for ws, n, want in ((None, need, bad), (BASE + 8 * (1 << 40), need - 1, bad),
                        (BASE + 8 * (1 << 40) + 512, need, L.FSDP_ERR_ALIGNMENT),
                        (BASE + 5 * (1 << 40), need, bad)):  # the workspace over a gradient
        assert lib.fsdp_head_loss(ctypes.byref(a), ws, n, None) == want


def arrays(addresses, numels, dtypes):
    n = max(len(addresses), len(numels), len(dtypes))
    return ((ctypes.c_void_p * max(n, 1))(*addresses), (ctypes.c_int64 * max(n, 1))(*numels),
            (ctypes.c_int32 * max(n, 1))(*dtypes))


def test_grad_norm_and_clip_refuse(lib, L):
    bad = L.FSDP_ERR_INVALID_ARG
    n = ctypes.c_int64(-1)
    p, num, dt = arrays([BASE, BASE + 4096], [100, 10], [L.FSDP_F32, L.FSDP_BF16])
    assert lib.fsdp_grad_norm_workspace(num, dt, 2, ctypes.byref(n)) == L.FSDP_OK and n.value > 0
    need, norm, ws = n.value, BASE + 8192, BASE + 16384

    def grad_norm(p=p, num=num, dt=dt, k=2, scale=1.0, norm=norm, ws=ws, nbytes=need):
        return lib.fsdp_grad_norm(p, num, dt, k, scale, norm, ws, nbytes, None)

    assert grad_norm(k=-1) == bad and grad_norm(p=None) == bad and grad_norm(num=None) == bad
    assert grad_norm(scale=float("nan")) == bad and grad_norm(norm=None) == bad and grad_norm(ws=None) == bad
    assert grad_norm(nbytes=need - 1) == bad
    assert grad_norm(norm=norm + 2) == L.FSDP_ERR_ALIGNMENT and grad_norm(ws=ws + 8) == L.FSDP_ERR_ALIGNMENT
    assert grad_norm(norm=ws + 8) == bad and grad_norm(norm=BASE + 40) == bad and grad_norm(ws=BASE) == bad
    assert grad_norm(p=arrays([BASE, None], [100, 10], [0, 1])[0]) == bad
    assert grad_norm(p=arrays([BASE + 2, BASE + 4096], [100, 10], [0, 1])[0]) == L.FSDP_ERR_ALIGNMENT
    assert grad_norm(num=arrays([], [100, -1], [])[1]) == bad
    assert grad_norm(dt=arrays([], [], [0, 5])[2]) == L.FSDP_ERR_UNSUPPORTED_DTYPE
    assert lib.fsdp_grad_norm_workspace(num, dt, 2, None) == bad

    def clip(src=p, dst=p, norm=norm, max_norm=1.0, scale=1.0):
        return lib.fsdp_clip_grads(src, dst, num, dt, 2, norm, max_norm, scale, None)

    for m in (0.0, -1.0, float("nan")):
        assert clip(max_norm=m) == bad
    assert clip(norm=None) == bad and clip(norm=norm + 1) == L.FSDP_ERR_ALIGNMENT and clip(scale=float("inf")) == bad
    assert clip(dst=None) == bad
    assert clip(dst=arrays([BASE, BASE + 392], [], [])[0]) == bad       # two results overlap
    assert clip(dst=arrays([BASE + 4, BASE + 4096], [], [])[0]) == bad  # shifted over its own source
    assert clip(dst=arrays([BASE + 4096, BASE + 1024], [], [])[0]) == bad  # over another's source
    assert clip(dst=arrays([norm, BASE + 4096], [], [])[0]) == bad      # over the norm


def test_clip_plans_refuse(lib, L):
    bad = L.FSDP_ERR_INVALID_ARG
    n, plan = ctypes.c_int64(-1), ctypes.c_void_p(None)
    cfg = L.FsdpStepConfig(L.FSDP_OPT_SGD, L.FSDP_F32, 1e-3, 0.9, 0.95, 1e-8, 0.0, 1, 1.0)
    # no units: an empty model is fine, its size only the counter's
    assert lib.fsdp_clip_plan_workspace(None, 0, ctypes.byref(n)) == L.FSDP_OK and n.value >= 4
    assert lib.fsdp_clip_plan_workspace(None, 1, ctypes.byref(n)) == bad
    assert lib.fsdp_clip_plan_workspace(None, 0, None) == bad
    assert lib.fsdp_clip_plan_workspace_ex(None, 0, ctypes.byref(cfg), ctypes.byref(n)) == L.FSDP_OK
    assert lib.fsdp_clip_plan_workspace_ex(None, 0, None, ctypes.byref(n)) == bad
    assert lib.fsdp_clip_plan_create(None, 0, 1, None, 0, None, None, ctypes.byref(plan)) == bad
    assert lib.fsdp_clip_plan_create(None, 0, 1, BASE + 16, 1 << 20, None, None,
                                     ctypes.byref(plan)) == L.FSDP_ERR_ALIGNMENT
    assert lib.fsdp_clip_plan_create(None, 0, -1, BASE, 1 << 20, None, None, ctypes.byref(plan)) == bad
    assert lib.fsdp_clip_plan_create(None, 0, 1, BASE, 8, None, None, ctypes.byref(plan)) == bad
    assert lib.fsdp_clip_plan_create(None, 0, 1, BASE, 1 << 20, None, None, None) == bad
    cfg.reduce_dtype = L.FSDP_BF16
    assert lib.fsdp_clip_plan_create_ex(None, 0, ctypes.byref(cfg), 1, BASE, 1 << 20, None, None,
                                        ctypes.byref(plan)) == L.FSDP_ERR_UNSUPPORTED_DTYPE
    assert not plan
    hp = L.FsdpAdamwHparams(1e-3, 0.9, 0.95, 1e-8, 0.0, 1, 1.0)
    assert lib.fsdp_clip_plan_launch(None, ctypes.byref(hp), 1.0, BASE, None) == bad
    assert lib.fsdp_clip_plan_launch_ex(None, ctypes.byref(cfg), 1.0, BASE, None) == bad
    assert lib.fsdp_clip_plan_destroy(None) == L.FSDP_OK
    # an empty model's plan: refused scalars, the wrong kind of launch
    assert lib.fsdp_clip_plan_create(None, 0, 1, BASE, 1 << 20, None, None, ctypes.byref(plan)) == L.FSDP_OK
    for m in (0.0, -1.0, float("nan")):
        assert lib.fsdp_clip_plan_launch(plan, ctypes.byref(hp), m, BASE, None) == bad
    assert lib.fsdp_clip_plan_launch(plan, None, 1.0, BASE, None) == bad
    assert lib.fsdp_clip_plan_launch(plan, ctypes.byref(hp), 1.0, None, None) == bad
    assert lib.fsdp_clip_plan_launch(plan, ctypes.byref(hp), 1.0, BASE + 2, None) == L.FSDP_ERR_ALIGNMENT
    hp.step = 0
    assert lib.fsdp_clip_plan_launch(plan, ctypes.byref(hp), 1.0, BASE, None) == bad
    assert lib.fsdp_clip_plan_launch_ex(plan, ctypes.byref(cfg), 1.0, BASE, None) == bad
    assert lib.fsdp_clip_plan_destroy(plan) == L.FSDP_OK


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    import torch
    import sharded_fsdp_reduce_gb300 as F
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        F.fsdp_head_loss(x, torch.zeros(10, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64), torch.zeros(()))
    with pytest.raises(ValueError):
        F.GradClip([x])
    with pytest.raises(ValueError):
        F.GradClip([x], out=[])
    with pytest.raises(TypeError):
        F.HeadLoss(10, 8, torch.float64, 4)
    with pytest.raises(ValueError):
        F.HeadLoss(10, 8, torch.bfloat16, 4, reduction="none")


def test_workspace_memory_at_any_base():
    """The memory is found at its alignment wherever the allocator's block begins."""
    from sharded_fsdp_reduce_gb300.workspace import take
    held = []
    for n in (0, 1, 100, 4096, 70_001):
        for k in range(8):
            buf = take(n, "cpu", alignment=1024, zeroed=k % 2 == 0)
            assert buf.numel() == n and (n == 0 or buf.data_ptr() % 1024 == 0)
            assert k % 2 or not bool(buf.any())
            assert take(n, "cpu", zeroed=True).numel() == n
            held.append((buf, bytearray(100 + 16 * k)))


def test_a_workspace_of_another_device_is_refused(monkeypatch):
    """An object made on one GPU and called with another one current, its
    tensors there: the workspace would reach the kernels as a foreign address."""
    import types
    import torch
    from sharded_fsdp_reduce_gb300.workspace import Workspace
    ws = Workspace.__new__(Workspace)
    ws.buf, ws._device, ws._made_on, ws._ready, ws._in_capture = torch.zeros(8), 0, 5, None, False
    s = types.SimpleNamespace(cuda_stream=5)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert ws.on(s) is s
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        ws.on(s)
