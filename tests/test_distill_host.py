"""Host-side checks of the distillation loss's entry points: workspace sizes and
refusals, with no GPU and nothing enqueued (the addresses are made up and never
read)."""
import ctypes

import pytest

BASE = 1 << 44  # a made-up device address, 16-byte aligned
STEP = 1 << 40


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


def args(L, T=100, V=1000, D=64, K=20, dtype=None, grad=True, **kw):
    a = L.FsdpHeadDistillArgs()
    a.dtype = L.FSDP_BF16 if dtype is None else dtype
    a.teacher_dtype, a.id_bits, a.temperature, a.grad_scale = L.FSDP_F32, 64, 2.0, 1.0
    a.tokens, a.vocab, a.dim, a.top = T, V, D, K
    a.hidden, a.weight, a.teacher_logits, a.teacher_ids, a.loss, a.token_loss = (BASE + k * STEP for k in range(6))
    if grad:
        a.d_hidden, a.d_weight = BASE + 6 * STEP, BASE + 7 * STEP
    a.ld_hidden = a.ld_weight = a.ld_d_hidden = a.ld_d_weight = D
    a.ld_teacher_logits = a.ld_teacher_ids = K
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def workspace(lib, a):
    n = ctypes.c_int64(-1)
    return lib.fsdp_head_distill_workspace(ctypes.byref(a), ctypes.byref(n)), n.value


def test_workspace(lib, L):
    st, grad = workspace(lib, args(L, T=1000, V=50257, D=768))
    assert st == L.FSDP_OK and grad >= 2 * 1000 * 50257  # the 16-bit exponentials of one band
    st, losses = workspace(lib, args(L, T=1000, V=50257, D=768, grad=False))
    assert st == L.FSDP_OK and losses < grad // 4
    # an entry takes 16 bytes of a row
    st, more = workspace(lib, args(L, T=1000, V=50257, D=768, K=120, ld_teacher_logits=120, ld_teacher_ids=120))
    assert st == L.FSDP_OK and abs(more - grad - 16 * 1000 * 100) < 1 << 14
    # bands bound the exponentials whatever the tokens
    st, long = workspace(lib, args(L, T=1_000_000, V=128_000, D=64))
    assert st == L.FSDP_OK and long < (4 << 30) * 1.5 + 4 * 128_000 * 64 + 48 * 1_000_000
    assert workspace(lib, args(L, T=0)) == (L.FSDP_OK, 0)


@pytest.mark.parametrize("T,V,D,K,dtype,band", [
    (3000, 1003, 200, 64, "f16", 0), (700, 5003, 768, 256, "f32", 0), (30, 33, 8, 5, "f32", 0), (9, 40, 72, 1, "bf16", 0),
    (900, 700, 64, 10, "bf16", 100), (70_000, 131_072, 64, 8, "bf16", 0),
])
@pytest.mark.parametrize("grad", [True, False])
def test_workspace_is_enough_for_every_shorter_call(lib, L, T, V, D, K, dtype, band, grad):
    code = dict(f32=L.FSDP_F32, bf16=L.FSDP_BF16, f16=L.FSDP_F16)[dtype]
    kw = dict(V=V, D=D, dtype=code, band=band, grad=grad)
    st, most = workspace(lib, args(L, T=T, K=K, **kw))
    assert st == L.FSDP_OK
    for t in list(range(1, min(T, 600))) + list(range(600, T, max(1, T // 1000))):
        for k in {1, K}:
            st, n = workspace(lib, args(L, T=t, K=k, **kw))
            assert st == L.FSDP_OK and n <= most, (t, k, n, most)


def test_refusals(lib, L):
    bad, off = L.FSDP_ERR_INVALID_ARG, L.FSDP_ERR_ALIGNMENT
    cases = [
        (dict(dtype=7), L.FSDP_ERR_UNSUPPORTED_DTYPE), (dict(teacher_dtype=3), L.FSDP_ERR_UNSUPPORTED_DTYPE),
        (dict(id_bits=16), L.FSDP_ERR_UNSUPPORTED_DTYPE),
        (dict(tokens=-1), bad), (dict(vocab=0), bad), (dict(dim=0), bad), (dict(tokens=1 << 40), bad),
        (dict(top=0), bad), (dict(top=1025, ld_teacher_logits=1025, ld_teacher_ids=1025), bad),
        (dict(temperature=0.0), bad), (dict(temperature=-1.0), bad), (dict(temperature=float("nan")), bad),
        (dict(temperature=float("inf")), bad), (dict(temperature=1e-4), bad),
        (dict(band=-1), bad), (dict(reduction=2), bad), (dict(reserved=1), bad), (dict(grad_scale=float("nan")), bad),
        (dict(grad_scale=3e38), bad),  # times the temperature it is infinite
        (dict(hidden=None), bad), (dict(weight=None), bad), (dict(teacher_logits=None), bad),
        (dict(teacher_ids=None), bad), (dict(loss=None), bad),
        (dict(ld_hidden=63), bad), (dict(ld_weight=0), bad), (dict(ld_teacher_logits=19), bad),
        (dict(ld_teacher_ids=19), bad), (dict(ld_teacher_ids=1 << 50), bad),
        (dict(tokens=1 << 30, ld_teacher_ids=1 << 34), bad), (dict(tokens=1 << 29, ld_teacher_logits=1 << 33), bad),
        (dict(hidden=BASE + 1), off), (dict(teacher_logits=BASE + 2 * STEP + 2), off),
        (dict(teacher_ids=BASE + 3 * STEP + 4), off), (dict(loss=BASE + 4 * STEP + 2), off),
        (dict(wait_timeouts=BASE + 2), off),
        (dict(d_hidden=BASE), bad), (dict(d_weight=BASE + STEP + 128), bad), (dict(d_hidden=BASE + 7 * STEP), bad),
        (dict(d_weight=BASE + 2 * STEP), bad), (dict(loss=BASE + 3 * STEP), bad), (dict(token_loss=BASE + 2 * STEP), bad),
        (dict(loss=BASE + 5 * STEP), bad),
    ]
    for kw, want in cases:
        assert workspace(lib, args(L, **kw))[0] == want, kw
        assert lib.fsdp_head_distill(ctypes.byref(args(L, **kw)), BASE + 8 * STEP, 1 << 40, None) == want, kw
    assert lib.fsdp_head_distill(None, BASE, 1 << 40, None) == bad
    a = args(L)
    assert lib.fsdp_head_distill_workspace(ctypes.byref(a), None) == bad
    _, need = workspace(lib, a)
    for k in (0, 1, 2, 3, 5, 6, 7):  # the workspace over a buffer of the call
        assert lib.fsdp_head_distill(ctypes.byref(a), BASE + k * STEP, 1 << 40, None) == bad, k
    for ws, n, want in ((None, need, bad), (BASE + 8 * STEP, need // 2, bad), (BASE + 8 * STEP + 512, need, off)):
        assert lib.fsdp_head_distill(ctypes.byref(a), ws, n, None) == want
    assert workspace(lib, args(L, id_bits=32, teacher_ids=BASE + 3 * STEP + 4))[0] == L.FSDP_OK
