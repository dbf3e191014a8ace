"""Many new tokens over the 8-bit paged cache where the library writes the codes' rows out first: as near to the
definition with the default workspace as on the codes themselves."""

import pytest
import torch

import sparse_attention_kv_dsa_gb300.echo as E

from paged_q8_ref import F8, PagedQ8, attend_q8
from paged_ref import DEV, check_rows, half_step

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def starts(new):
    return torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("cap", [0.0, 6.0])
@pytest.mark.parametrize("d,Hq,Hkv,lens,new", [(128, 8, 2, [700], [400]), (64, 16, 2, [300, 420], [300, 130]), (64, 2, 1, [1100], [1100])])
def test_default_workspace_keeps_float16_weights(d, Hq, Hkv, lens, new, cap, alibi):
    """Every value row is one row u under a sign and a row sees two tokens: half of the results are u times a difference
    of two weights, so that what the weights were rounded to shows beside the rounding of the result.  The bound
    is that of float16 weights: their half step, 2^-11 of sum p|v|, what attend_q8 has for float32, and half of
    bf16's step at the result (2^-8 below its power of two), for which attend_q8 takes half a step of its value."""
    N, B, scale = sum(new), len(lens), 0.6
    P = PagedQ8(lens, 16, Hkv, d, seed=d, exps=(-6, -6))
    assert E.paged_prefill_q8_workspace_bytes(N, B, Hq, Hkv, d, P.table.shape[1], 16) > E.paged_prefill_workspace_bytes(N, B, Hq, Hkv, d)
    g = torch.Generator().manual_seed(d)
    u = torch.randint(0x30, 0x78, (d,), generator=g, dtype=torch.uint8)
    for b, n in enumerate(lens):
        sign = torch.randint(0, 2, (n, Hkv, 1), generator=g)
        pg, row = P.at(b, torch.arange(n))
        P.vc[pg, row] = (u + 128 * sign).to(torch.uint8).to(DEV)
        P.V[b] = (1.0 - 2.0 * sign) * u.view(F8).double() * 2.0 ** -6
    q = (torch.randn(N, Hq, d, generator=g) * d ** -0.5).to(BF).to(DEV)    # scores of a spread of some 1
    slopes = torch.full((Hq,), 0.25) if alibi else None
    out, lse = E.paged_attn_prefill(q, starts(new), *P.pages, P.table, P.seq_len, scale, softcap=cap, window=2,
                                    slopes=slopes.to(DEV) if alibi else None, status=P.status, **P.scales)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    r = 0
    for b, n in enumerate(new):
        s, L = slice(r, r + n), lens[b]
        want, wlse, tol, ltol = attend_q8(q[s].double().cpu(), P.K[b], P.V[b], P.VE[b], torch.arange(L - n, L), scale, cap=cap,
                                          window=2, slopes=slopes)
        have, off = out[s].double().cpu(), tol - 1.01 * half_step(BF) * want.abs()
        step = torch.exp2(torch.floor(torch.log2(torch.maximum(have.abs(), want.abs()).clamp(min=1e-30))) - 8)
        worst = ((have - want).abs() - 1.01 * step - off).max().item()
        assert worst <= 0, f"sequence {b}: {worst} past the bound"
        assert torch.all((lse[s].double().cpu() - wlse).abs() <= ltol)
        r += n


@pytest.mark.parametrize("kw", [dict(window=64), dict(window=64, prefix=40), dict(window=300, first=19700), dict(first=19500),
                                dict(first=19500, prefix=19530), dict(window=1)])
@pytest.mark.parametrize("T,d", [(16, 128), (24, 64), (1000, 64)])
def test_only_tokens_that_a_row_sees_are_written_out(T, d, kw):
    """Many rows at the end of a long cache that see a few of its tokens: the others are not read (NaN codes under a NaN
    exponent, no page for most) and leave their places in the workspace alone."""
    L, n, Hq, Hkv, u8 = 20000, 200, 16, 2, torch.uint8
    P = PagedQ8([L], T, Hkv, d, seed=T)
    first, window, prefix = kw.get("first"), kw.get("window", 0), kw.get("prefix", 0)
    t, p = torch.arange(L), torch.arange(L - n, L)[:, None]
    see = (t <= p) & (t > p - window if window else t >= 0) | (t < prefix)
    see = (see & (t >= (first or 0))).any(0)
    pg, row = P.at(0, t[~see])
    for pool, x in ((P.kc, 0x7f), (P.vc, 0xff), (P.ke, 255), (P.ve, 255)):
        pool[pg, row] = x
    table = P.table.clone()
    for i in range(-(-L // T)):
        if not see[i * T:(i + 1) * T].any():
            table[0, i] = -1
    q = (torch.randn(n, Hq, d, generator=torch.Generator().manual_seed(1)) * 0.1).to(BF).to(DEV)
    first_tok = None if first is None else torch.full((n,), first, dtype=torch.int32, device=DEV)
    small = -(-E.paged_prefill_workspace_bytes(n, 1, Hq, Hkv, d) // 256) * 256
    ws = torch.full((E.paged_prefill_q8_workspace_bytes(n, 1, Hq, Hkv, d, table.shape[1], T),), 0xa5, dtype=u8, device=DEV)
    rows = 2 * (-(-table.shape[1] * T * Hkv * d * 2 // 256) * 256)
    assert ws.numel() >= small + rows
    out, lse = E.paged_attn_prefill(q, starts([n]), *P.pages, table, P.seq_len, 0.1, window=window, first_tok=first_tok,
                                    prefix_len=torch.tensor([prefix], dtype=torch.int32, device=DEV) if prefix else None,
                                    workspace=ws, status=P.status, **P.scales)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    check_rows("rows", out, lse, attend_q8(q.double().cpu(), P.K[0], P.V[0], P.VE[0], torch.arange(L - n, L), 0.1, window=window,
                                           first=None if first is None else [first] * n, prefix=prefix))
    written = int((ws[small:small + rows] != 0xa5).sum())
    assert 0.9 <= written / (int(see.sum()) * Hkv * d * 2 * 2) <= 1


def test_rows_written_out_stay_below_a_gibibyte():
    base = E.paged_prefill_workspace_bytes(8192, 1, 64, 8, 128)
    for tokens, more in ((16, True), (1 << 18, True), ((1 << 18) + 16, False), (1 << 20, False)):
        size = E.paged_prefill_q8_workspace_bytes(8192, 1, 64, 8, 128, tokens // 16, 16)
        assert (size > base) == more and size <= base + 512 + (1 << 30) + tokens // 4
