"""The token embedding where its kernels change form: what a lookup reads at a
table's end, the edges of the sorts, windows of rows that no token uses."""

import pytest
import torch

from test_embedding_gpu import DEV, DT, F, IGNORE, check_lookup, inputs  # noqa: F401 (F: a fixture)

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
