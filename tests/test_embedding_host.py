"""Host-side checks of the token embedding's entry points: workspace sizes and
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


def lookup_args(L, T=100, V=1000, D=64, **kw):
    a = L.FsdpEmbedArgs()
    a.dtype, a.count, a.vocab, a.dim, a.ignore_index, a.scale = L.FSDP_BF16, T, V, D, -100, 1.0
    a.tokens, a.weight, a.out = BASE, BASE + STEP, BASE + 2 * STEP
    a.ld_weight = a.ld_out = D
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def grad_args(L, T=100, V=1000, D=64, **kw):
    a = L.FsdpEmbedGradArgs()
    a.dtype, a.count, a.vocab, a.dim, a.ignore_index, a.scale = L.FSDP_BF16, T, V, D, -100, 1.0
    a.tokens, a.d_out, a.d_weight = BASE, BASE + STEP, BASE + 2 * STEP
    a.ld_d_out = a.ld_d_weight = D
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def workspace(lib, a):
    n = ctypes.c_int64(-1)
    st = lib.fsdp_embed_grad_workspace(ctypes.byref(a), ctypes.byref(n))
    return st, n.value


def test_workspace(lib, L):
    st, n = workspace(lib, grad_args(L, T=10_000, V=50257, D=768))
    # the sorted tokens and their places, twice, and no more than two fp32 rows of eight tokens
    assert st == L.FSDP_OK and 16 * 10_000 <= n <= 16 * 10_000 + 2 * 4 * 768 * 1250 + 5 * 256
    assert workspace(lib, grad_args(L, T=0)) == (L.FSDP_OK, 0)
    assert workspace(lib, grad_args(L, T=0, tokens=None, d_out=None)) == (L.FSDP_OK, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(300, 64), (5000, 8192), (70_000, 768), (70_000, 100)])
def test_workspace_is_enough_for_every_shorter_call(lib, L, T, D, dtype):
    code = dict(f32=L.FSDP_F32, bf16=L.FSDP_BF16)[dtype]
    st, most = workspace(lib, grad_args(L, T=T, D=D, dtype=code))
    assert st == L.FSDP_OK
    for t in list(range(1, min(T, 3000))) + list(range(3000, T, 97)):
        # (at any address and stride)
        for kw in (dict(), dict(d_out=BASE + STEP + 4), dict(d_weight=BASE + 2 * STEP + 4), dict(ld_d_out=D + 3)):
            st, n = workspace(lib, grad_args(L, T=t, D=D, dtype=code, **kw))
            assert st == L.FSDP_OK and n <= most, (t, kw, n, most)


def test_refusals(lib, L):
    bad, off = L.FSDP_ERR_INVALID_ARG, L.FSDP_ERR_ALIGNMENT
    common = [
        (dict(dtype=7), L.FSDP_ERR_UNSUPPORTED_DTYPE),
        (dict(count=-1), bad), (dict(count=1 << 31), bad), (dict(vocab=0), bad), (dict(vocab=1 << 31), bad),
        (dict(dim=0), bad), (dict(scale=float("inf")), bad), (dict(scale=float("nan")), bad),
        (dict(tokens=None), bad), (dict(tokens=BASE + 4), off),
    ]
    for kw, want in common + [
        (dict(weight=None), bad), (dict(out=None), bad), (dict(ld_weight=63), bad), (dict(ld_out=63), bad),
        (dict(ld_out=1 << 50), bad), (dict(weight=BASE + STEP + 1), off), (dict(out=BASE + 2 * STEP + 1), off),
        (dict(out=BASE + STEP + 128), bad), (dict(out=BASE), bad), (dict(reserved=1), bad),
    ]:
        assert lib.fsdp_embed(ctypes.byref(lookup_args(L, **kw)), None) == want, kw
    assert lib.fsdp_embed(None, None) == bad
    for kw, want in common + [
        (dict(d_out=None), bad), (dict(d_weight=None), bad), (dict(ld_d_out=63), bad), (dict(ld_d_weight=0), bad),
        (dict(ld_d_weight=1 << 50), bad), (dict(d_out=BASE + STEP + 1), off), (dict(d_weight=BASE + 2 * STEP + 1), off),
        (dict(d_weight=BASE + STEP + 128), bad), (dict(d_weight=BASE - 128), bad), (dict(accumulate=2), bad),
        (dict(accumulate=-1), bad),
    ]:
        assert workspace(lib, grad_args(L, **kw))[0] == want, kw
        assert lib.fsdp_embed_grad(ctypes.byref(grad_args(L, **kw)), BASE + 3 * STEP, 1 << 30, None) == want, kw
    assert lib.fsdp_embed_grad(None, BASE, 1 << 30, None) == bad
    a = grad_args(L)
    assert lib.fsdp_embed_grad_workspace(ctypes.byref(a), None) == bad
    _, need = workspace(lib, a)
    for ws, n, want in ((None, need, bad), (BASE + 3 * STEP, need - 1, bad), (BASE + 3 * STEP + 128, need, off),
                        (BASE, need, bad), (BASE + STEP, need, bad), (BASE + 2 * STEP, need, bad)):
        assert lib.fsdp_embed_grad(ctypes.byref(a), ws, n, None) == want, ws
