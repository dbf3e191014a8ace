"""The buffers that the paged calls make where the caller gives none are torch's own: dispatch modes see them, and
they are filled where torch is asked to fill what is new."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import sparse_attention_kv_dsa_gb300.echo as E

from paged_q8_ref import PagedQ8
from paged_ref import DEV, Paged

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def pool(q8):
    if q8:
        P = PagedQ8([200, 40], 16, 2, 64)
        return (*P.pages, P.table, P.seq_len), P.scales
    P = Paged([200, 40], 16, 2, 64, BF)
    return (P.k, P.v, P.table, P.seq_len), {}


class Made(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func.overloadpacket in (torch.ops.aten.empty, torch.ops.aten.empty_strided, torch.ops.aten.empty_like, torch.ops.aten.new_empty):
            self.shapes.append((tuple(out.shape), out.dtype))
        return out


@pytest.mark.parametrize("q8", [False, True])
def test_dispatch_modes_see_the_buffers(q8):
    args, kw = pool(q8)
    q, rows = (torch.zeros(n, 4, 64, dtype=BF, device=DEV) for n in (2, 6))
    qs = torch.tensor([0, 4, 6], dtype=torch.int32, device=DEV)
    for call, n in ((lambda: E.paged_attn_decode(q, *args, 0.1, **kw), 2), (lambda: E.paged_attn_prefill(rows, qs, *args, 0.1, **kw), 6)):
        with Made() as made:
            call()
        assert made.shapes[:2] == [((n, 4, 64), BF), ((n, 4), torch.float32)] and made.shapes[2][1] == torch.uint8


@pytest.mark.parametrize("q8", [False, True])
def test_buffers_are_filled_where_torch_fills_new_memory(q8):
    args, kw = pool(q8)
    rows = torch.zeros(6, 4, 64, dtype=BF, device=DEV)
    qs = torch.tensor([0, 3, 4], dtype=torch.int32, device=DEV)        # two rows behind the last sequence
    before = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = True
        for _ in range(3):
            junk = torch.full((1 << 20,), 3.0, device=DEV)
            del junk
            out, lse = E.paged_attn_prefill(rows, qs, *args, 0.1, **kw)
            assert bool(out[4:].isnan().all()) and bool(lse[4:].isnan().all()) and bool(out[:4].isfinite().all())
    finally:
        torch.use_deterministic_algorithms(before[0])
        torch.utils.deterministic.fill_uninitialized_memory = before[1]
