"""Paged-cache calls as programs make them beside other work: many small calls one after the
other, calls on a stream of their own, batches padded with rows that see nothing."""

import pytest
import torch

import sparse_attention_kv_dsa_gb300.echo as E

from paged_ref import DEV, Paged, attend, check_rows

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------ many small calls --
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [1, 2, 17, 128, 129, 1000])
def test_decode_small_calls_give_the_same_bits_every_time(dtype, d, B):
    """Every warp of a CTA has to agree on where the CTA's run begins, whichever of them is
    first: 600 calls a case (14,400 in all), each behind another kernel that takes the
    instruction caches, bit for bit the first one's results."""
    Hq, Hkv, T = 8, 2, 16
    lens = [(29 * i) % 150 for i in range(1, B + 1)]
    P = Paged(lens, T, Hkv, d, dtype, seed=B)
    g = torch.Generator().manual_seed(B + 1)
    q = torch.randn(B, Hq, d, generator=g).to(dtype).to(DEV)
    ws = torch.empty(E.paged_decode_workspace_bytes(Hq, Hkv, d), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, Hq, device=DEV)
    call = lambda: E.paged_attn_decode(q, P.k, P.v, P.table, P.seq_len, 0.1, out=out, lse=lse, workspace=ws,  # noqa: E731
                                       status=P.status)
    call()
    torch.cuda.synchronize()
    for b in range(0, B, max(1, B // 5)):
        check_rows(f"sequence {b} of {B}", out[b:b + 1], lse[b:b + 1],
                   attend(q[b:b + 1].double().cpu(), P.K[b], P.V[b], [lens[b] - 1], 0.1, dtype=dtype))
    want, wlse = out.clone(), lse.clone()
    other = torch.zeros(1 << 16, device=DEV)
    bad = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(600):
        out.fill_(7.0)
        lse.fill_(7.0)
        if i % 4 == 0:
            other.sin_() if i % 8 else other.sort()
        call()
        bad += (out != want).sum() + (lse != wlse).sum()
    assert bad.item() == 0 and P.status.item() == E.OK
