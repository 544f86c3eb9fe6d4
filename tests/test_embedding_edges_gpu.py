"""The token embedding where its kernels change form: what a lookup reads at a
table's end, the edges of the sorts, windows of rows that no token uses."""
import math

import pytest
import torch

from test_embedding_gpu import DEV, DT, F, IGNORE, check_gradient, check_lookup, inputs  # noqa: F401 (F: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [1, 2, 5, 63, 66, 771])
@pytest.mark.parametrize("out_off", [0, 1])
@pytest.mark.parametrize("lead", [0, 1, 3])
def test_lookup_of_a_table_that_ends_its_buffer(F, D, out_off, lead, dt):
    """16-bit rows at every alignment of both sides; the last row's last element
    is the buffer's last."""
    V, T = 37, 70
    tokens, w0, _ = inputs(T, V, D, dt, "holes", seed=D)
    tokens[::5] = V - 1
    table = torch.empty(lead + V * D, dtype=DT[dt], device=DEV)
    w = table[lead:].view(V, D)
    w.copy_(w0)
    buf = torch.full((out_off + T * D + 3,), 7.0, dtype=DT[dt], device=DEV)
    out = buf[out_off:out_off + T * D].view(T, D)
    F.Embedding(V, D, DT[dt], T, grad=False).forward(tokens, w, out=out)
    check_lookup(out, tokens, w0, dt)
    assert bool((buf[:out_off] == 7).all()) and bool((buf[out_off + T * D:] == 7).all())


def check_exact(F, T, V, kind="skewed", ignored=0.1):
    """Integers of few bits add up exactly in any order: which rows add up shows."""
    g = torch.Generator(device=DEV).manual_seed(T)
    if kind == "skewed":
        u = torch.rand(T, device=DEV, dtype=torch.float64, generator=g)
        tokens = (torch.exp(u * math.log(V + 1.0)).long() - 1).clamp_(0, V - 1)
    else:
        tokens = torch.randint(0, V, (T,), device=DEV, generator=g)
    tokens[:2] = torch.tensor([V - 1, 0], device=DEV)[:T]
    tokens[2:][torch.rand(T - 2, device=DEV, generator=g) < ignored] = IGNORE
    dy = torch.randint(-8, 9, (T, 4), device=DEV, generator=g).float()
    live = tokens != IGNORE
    want = torch.zeros(V, 4, dtype=torch.float64, device=DEV).index_put_((tokens[live],), dy[live].double(),
                                                                        accumulate=True)
    dw = torch.full((V, 4), float("nan"), device=DEV)
    F.fsdp_embed_grad(tokens, dy, dw)
    assert torch.equal(dw.double(), want)
    dw = torch.ones(V, 4, device=DEV)
    F.fsdp_embed_grad(tokens, dy, dw, accumulate=True)
    assert torch.equal(dw.double(), want + 1)


# One digit, two (of 7 and of 9 bits) and three; counted up to 4096 tokens (below
# 2^20), in the shared memory of 8 CTAs up to 32768 and of 16 up to 65536, then
# through memory.
@pytest.mark.parametrize("T", [4095, 4096, 4097, 8192, 8193, 16385, 32767, 32768, 32769, 40001, 50000, 65535, 65536,
                               65537, 70000, 140000])
@pytest.mark.parametrize("V", [1000, 1024, 1 << 14, 1 << 17, (1 << 20) + 5])
def test_the_sort_at_the_edges_of_its_forms(F, T, V):
    for kind in ("skewed", "uniform"):
        check_exact(F, T, V, kind)


@pytest.mark.parametrize("V", [(1 << 20) - 2, (1 << 20) - 1, 1 << 20, (1 << 20) + 1])
@pytest.mark.parametrize("T", [2, 129, 4095, 4096])
def test_the_largest_vocabulary_that_is_placed_by_counting(F, T, V):
    """The key that stands for no token is the vocabulary's size: 20 bits of it
    fit beside the position."""
    check_exact(F, T, V, "uniform", ignored=0.4)


@pytest.mark.parametrize("T,V", [(70000, (1 << 20) + 5), (40000, (1 << 20) + 5), (50001, 3000), (65536, 50257)])
def test_long_batches_have_the_same_bits_every_time(F, T, V):
    tokens, w, dy = inputs(T, V, 24, "bf16", "skewed", seed=1)
    table = F.Embedding(V, 24, torch.bfloat16, T)
    first = table.backward(tokens, dy, torch.empty_like(w))
    for _ in range(3):
        assert torch.equal(table.backward(tokens, dy, torch.empty_like(w)), first)
    check_gradient(first, tokens, dy, "bf16")


@pytest.mark.parametrize("T", [31, 32, 33, 100, 1000])
@pytest.mark.parametrize("D", [1, 2, 31, 33, 63, 64, 65, 257])
def test_lookup_of_short_fp32_rows_at_any_alignment(F, T, D):
    tokens, w0, _ = inputs(T, 90, D, "f32", "holes", seed=D)
    buf = torch.empty(1 + 90 * D, device=DEV)
    w = buf[1:].view(90, D)
    w.copy_(w0)
    out = torch.full((T * D + 2,), 7.0, device=DEV)
    F.Embedding(90, D, torch.float32, T, scale=1.5, grad=False).forward(tokens, w, out=out[1:1 + T * D].view(T, D))
    check_lookup(out[1:1 + T * D].view(T, D), tokens, w0, "f32", 1.5)
    assert float(out[0]) == 7 and float(out[-1]) == 7


@pytest.mark.parametrize("T", [0, 5, 3000])
def test_zeros_of_more_rows_than_a_window(F, T):
    """Three CTAs an SM have a stretch of the table each, and know the use of
    65536 rows at a time."""
    window = 3 * torch.cuda.get_device_properties(0).multi_processor_count * 65536
    V = window + window // 3 + 1001
    g = torch.Generator(device=DEV).manual_seed(T)
    tokens = torch.randint(0, V, (T,), device=DEV, generator=g)
    if T:  # stretches' and windows' ends
        each = -(-V // (window // 65536))
        tokens[:5] = torch.tensor([0, V - 1, each - 1, each, 65536], device=DEV)
    dy = torch.randint(1, 9, (T, 1), device=DEV, generator=g).to(torch.bfloat16)
    dw = torch.full((V, 1), float("nan"), dtype=torch.bfloat16, device=DEV)
    F.fsdp_embed_grad(tokens, dy, dw)
    want = torch.zeros(V, 1, device=DEV).index_put_((tokens,), dy.float(), accumulate=True)
    assert torch.equal(dw.float(), want)  # (a token's few single digits add up exactly in bf16)


def test_two_tables_at_once_on_two_streams(F):
    """Each with its own workspace, long and short calls side by side."""
    V, D = 5000, 72
    cases = [(3000, "skewed"), (50000, "uniform")]
    sets = [inputs(T, V, D, "bf16", kind, seed=k) for k, (T, kind) in enumerate(cases)]
    tables = [F.Embedding(V, D, torch.bfloat16, T) for T, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.empty(V, D, dtype=torch.bfloat16, device=DEV) for _ in range(6)] for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for k in range(6):
        for (tokens, _, dy), table, s, out in zip(sets, tables, streams, outs):
            table.backward(tokens, dy, out[k], stream=s)
    torch.cuda.synchronize()
    for (tokens, _, dy), out in zip(sets, outs):
        check_gradient(out[0], tokens, dy, "bf16")
        assert all(torch.equal(out[0], o) for o in out[1:])
