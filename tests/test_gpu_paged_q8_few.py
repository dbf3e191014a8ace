"""Many-token calls over the 8-bit paged cache with a few new tokens a sequence on average: batches of single tokens
beside chunks of prompts, whose sequences go by their own rows, and the calls' errors on both kernels that they
take, and on rows written out: q_start and lengths outside their range, bad pages, tokens that no row sees."""

import pytest
import torch

import sparse_attention_kv_dsa_gb300.echo as E

from paged_q8_ref import PagedQ8, attend_q8
from paged_ref import DEV, check_rows
from test_gpu_paged_q8 import _prefill, starts

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def kernels(new, G, N=None):
    """Which kernels a call's sequences take: 'few' the single-token split for all (up to 1024 packed rows), or 'split',
    that for sequences of up to 32 packed rows and the tensor cores for the others."""
    N = sum(new) if N is None else N
    assert N * G <= 32 * len(new)
    return "few" if N * G <= 1024 else "split"


# single tokens, a few drafted ones and none beside chunks
MIXED = ([1 + (13 * i) % 300 for i in range(150)] + [900, 290, 40, 64, 700, 5],
         [(1, 1, 2, 1, 4, 0)[i % 6] if (13 * i) % 300 >= 4 else 1 for i in range(150)] + [170, 33, 40, 0, 5, 3])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,T", [(8, 1, 16), (16, 2, 5), (9, 1, 64), (32, 4, 20), (5, 1, 8)])
def test_chunks_beside_single_tokens(d, Hq, Hkv, T):
    assert kernels(MIXED[1], Hq // Hkv, sum(MIXED[1]) + 2) == "split"
    _prefill(*MIXED, T, Hq, Hkv, d, seed=Hq + T, tail_rows=2, heads_first=T == 8, strided=Hq == 9)


@pytest.mark.parametrize("kw", [dict(cap=30.0), dict(cap=2.0, sharp=2.0), dict(alibi=True), dict(window=3), dict(window=100),
                                dict(prefix=[(7 * i) % 90 for i in range(156)]), dict(scale=-0.2), dict(scale=0.0),
                                dict(window=20, prefix=[(7 * i) % 90 for i in range(156)], alibi=True, cap=25.0),
                                dict(exps=(-15, 7), scale=2.0 ** -19)])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_beside_single_tokens_modifiers(kw, d):
    _prefill(*MIXED, 16, 8, 1, d, seed=3, **kw)


@pytest.mark.parametrize("new", [[4] * 32, [4] * 30 + [3, 5], [4] * 33, [4] * 36 + [3, 5], [0] * 39 + [129], [0] * 40 + [128], [33] + [1] * 140, [1] * 699 + [60, 0, 1]])
def test_borders_of_the_kernels_rows(new):
    """32 and 33 packed rows of a sequence and more, 1024 of a call and more, at 8 heads to a KV head."""
    N = max(sum(new), 100)
    assert kernels(new, 8, N) == ("few" if N <= 128 else "split")
    _prefill([n + 40 + 7 * (i % 5) for i, n in enumerate(new)], new, 16, 8, 1, 64, seed=7, tail_rows=N - sum(new))


def sizes(kind):
    """Sequences and new tokens of a call of 4 heads to a KV head on either kernel, with chunks among them on 'split', or
    of one whose codes are written out first."""
    lens, new = [200, 100, 90, 64, 300, 33], [4, 4, 2, 0, 8, 1]
    if kind == "rows":
        lens, new = [1000, 300, 90, 64, 300, 33], [1000, 250, 2, 0, 280, 8]
        assert sum(new) * 4 >= 1024 * len(new)
        return lens, new
    if kind == "split":
        lens, new = lens + [150, 260] + [40 + i % 9 for i in range(120)], new + [150, 60] + [1 + i % 3 for i in range(120)]
    assert kernels(new, 4) == kind
    return lens, new


def compare(P, q, new, out, lse, see=None, scale=0.02, but=None, **kw):
    """Every sequence (but one) against the definition over the tokens see[b] (all, where see is None)."""
    r = 0
    for b, n in enumerate(new):
        L = P.lens[b]
        if b == but:
            r += n
            continue
        k = torch.ones(L, dtype=torch.bool) if see is None else see[b]
        at = torch.cumsum(k.long(), 0)[L - n:] - 1 if L else torch.zeros(0)
        check_rows(f"sequence {b}: {n} of {L}", out[r:r + n], lse[r:r + n],
                   attend_q8(q[r:r + n].double().cpu(), P.K[b][k], P.V[b][k], P.VE[b][k], at, scale, **kw))
        r += n


@pytest.mark.parametrize("kind", ["few", "split", "rows"])
@pytest.mark.parametrize("d", [64, 128])
def test_starts_that_descend_write_nothing(kind, d):
    lens, new = sizes(kind)
    P = PagedQ8(lens, 16, 2, d, seed=3)
    N, B = sum(new), len(new)
    q = torch.randn(N, 8, d, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    good = starts(new).tolist()
    down, under, last = good[:], good[:], good[:]
    down[2], under[3], last[B] = N, -5, good[B - 1] - 1
    cases = [(down, E.ERR_INVALID_ARG), (under, E.ERR_INVALID_ARG), (last, E.ERR_INVALID_ARG), ([0] * (B + 1), E.OK), ([N] * (B + 1), E.OK),
             ([N + 100] * (B + 1), E.OK), ([-7] * (B + 1), E.OK)]
    for qs, code in cases:
        P.status.zero_()
        out, lse = torch.full_like(q, 7.0), torch.full((N, 8), 7.0, device=DEV)
        E.paged_attn_prefill(q, i32(qs), *P.pages, P.table, P.seq_len, 0.1, out=out, lse=lse, status=P.status, **P.scales)
        torch.cuda.synchronize()
        assert P.status.item() == code and bool((out == 7).all()) and bool((lse == 7).all()), qs
    # entries outside [0, N] are cut to it
    P.status.zero_()
    qs = [-3] + good[1:-1] + [N + 9]
    out, lse = E.paged_attn_prefill(q, i32(qs), *P.pages, P.table, P.seq_len, 0.02, status=P.status, **P.scales)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    compare(P, q, new, out, lse)


@pytest.mark.parametrize("kind", ["few", "split", "rows"])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_outside_their_range(kind, d):
    """A length past the page table is cut, a negative one is zero, and rows before position 0 see nothing; each is
    reported, and the other sequences' results stand.  On 'split' of sequence 0 (16 rows) and 6 (600)."""
    lens, new = sizes(kind)
    T, N = 16, sum(new)
    P = PagedQ8(lens, T, 2, d, seed=3)
    q = torch.randn(N, 8, d, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    qs = starts(new)
    cap = P.table.shape[1] * T
    for b in (0, 6) if kind == "split" else (0,):
        r = int(qs[b])
        for wrong in (cap + 5, -3, new[b] - 1):
            seq = P.seq_len.clone()
            seq[b] = wrong
            P.status.zero_()
            out, lse = E.paged_attn_prefill(q, qs, *P.pages, P.table, seq, 0.02, status=P.status, **P.scales)
            torch.cuda.synchronize()
            assert P.status.item() in ((E.ERR_INVALID_ARG, E.ERR_PAGE) if wrong > 0 else (E.ERR_INVALID_ARG,))
            L, m = min(max(wrong, 0), cap), new[b]
            none = max(0, m - L)                           # rows at negative positions
            assert not out[r:r + none].any() and bool(torch.isneginf(lse[r:r + none]).all())
            if L <= lens[b]:                               # (of a longer one, tokens that nobody wrote are seen: NaN)
                ref = attend_q8(q[r + none:r + m].double().cpu(), P.K[b][:L], P.V[b][:L], P.VE[b][:L], range(L - m + none, L), 0.02)
                check_rows(f"sequence {b} of {wrong}", out[r + none:r + m], lse[r + none:r + m], ref)
            compare(P, q, new, out, lse, but=b)


@pytest.mark.parametrize("kind", ["few", "split", "rows"])
@pytest.mark.parametrize("d,T", [(64, 16), (128, 8), (64, 5)])
def test_bad_pages_are_reported_and_their_tokens_skipped(kind, d, T):
    lens, new = sizes(kind)
    P = PagedQ8(lens, T, 2, d, seed=4)
    table, see = P.table.clone(), [torch.ones(n, dtype=torch.bool) for n in lens]
    for b, page, entry in ((0, 1, P.n_pages), (2, 0, -7), (4, 3, 1 << 30)) + (((6, 2, -1), (9, 1, P.n_pages + 5)) if kind == "split" else ()):
        table[b, page] = entry
        see[b][page * T:(page + 1) * T] = False
    q = torch.randn(sum(new), 8, d, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    out, lse = E.paged_attn_prefill(q, starts(new), *P.pages, table, P.seq_len, 0.02, status=P.status, **P.scales)
    torch.cuda.synchronize()
    assert P.status.item() == E.ERR_PAGE
    compare(P, q, new, out, lse, see)


@pytest.mark.parametrize("kind", ["few", "split", "rows"])
@pytest.mark.parametrize("d,T", [(64, 16), (128, 8), (64, 5)])
@pytest.mark.parametrize("kw", [dict(window=9), dict(window=30, prefix=12), dict()])
def test_tokens_that_no_row_sees_may_hold_anything(kind, d, T, kw):
    """Tokens below every row's window, and rows of the last page behind the sequence, are NaN codes under a NaN
    exponent; pages that hold nothing else are not in the table."""
    lens, new = sizes(kind)
    P = PagedQ8(lens, T, 2, d, seed=5)                     # (rows behind a sequence are NaN)
    window, prefix = kw.get("window", 0), kw.get("prefix", 0)
    table = P.table.clone()
    for b, (L, m) in enumerate(zip(lens, new)):
        t, p = torch.arange(L), torch.arange(L - m, L)[:, None]
        see = ((t <= p) & (t > p - window if window else t >= 0) | (t < prefix)).any(0)
        pg, row = P.at(b, t[~see])
        for pool, x in ((P.kc, 0x7f), (P.vc, 0xff), (P.ke, 255), (P.ve, 255)):
            pool[pg, row] = x
        for i in range(-(-L // T)):
            if not see[i * T:(i + 1) * T].any():
                table[b, i] = -1
    q = torch.randn(sum(new), 8, d, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    out, lse = E.paged_attn_prefill(q, starts(new), *P.pages, table, P.seq_len, 0.02, window=window,
                                    prefix_len=i32([prefix] * len(new)) if prefix else None, status=P.status, **P.scales)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    compare(P, q, new, out, lse, window=window, prefix=prefix)


def test_a_captured_batch_replayed_with_other_rows():
    """One graph for 300 packed rows of 100 sequences: single tokens, drafted ones, a chunk beside them, one sequence's
    alone, and no rows, each by q_start and lengths in device memory; and the same bits every time."""
    B, N, Hq, Hkv, d, T = 100, 300, 8, 1, 64, 16
    room = [400] * B
    P = PagedQ8(room, T, Hkv, d, seed=6)
    q = torch.randn(N, Hq, d, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    qs, seq = starts([1] * B), torch.full((B,), 300, dtype=torch.int32, device=DEV)
    ws = torch.empty(E.paged_prefill_workspace_bytes(N, B, Hq, Hkv, d), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(N, Hq, device=DEV)

    def call():
        E.paged_attn_prefill(q, qs, *P.pages, P.table, seq, 0.02, out=out, lse=lse, workspace=ws, status=P.status, **P.scales)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([1] * B, [3] * B, [1] * 60 + [200] + [1] * 39, [0] * 50 + [300] + [0] * 49, [5, 1] * 50, [0] * B):
        qs.copy_(starts(new))
        lens = [max(m, 100 + 3 * b) for b, m in enumerate(new)]
        seq.copy_(i32(lens))
        first = None
        for i in range(3):
            ws.fill_(255 * (i % 2))
            out.fill_(7.0)
            lse.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone(), lse.clone()
            first = first or got
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
        assert P.status.item() == E.OK
        r = 0
        for b, (n, L) in enumerate(zip(new, lens)):
            check_rows(f"sequence {b}: {n} of {L}", out[r:r + n], lse[r:r + n],
                       attend_q8(q[r:r + n].double().cpu(), P.K[b][:L], P.V[b][:L], P.VE[b][:L], range(L - n, L), 0.02))
            r += n
        assert bool((out[r:] == 7).all()) and bool((lse[r:] == 7).all())
