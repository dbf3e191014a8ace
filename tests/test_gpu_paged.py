"""The paged-cache calls against plain 64-bit forms: append with rotation, attention of one
new token, attention of many, each over head layouts, page sizes, types, lengths from zero
on, masks and modifiers; then together, captured, on other streams, and with bad pages."""

import math

import pytest
import torch

import sparse_attention_kv_dsa_gb300.echo as E

from paged_ref import DEV, Paged, attend, check_rows, cos_sin, doc_starts, half_step, rotate

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def starts(new):
    return torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------ append --
def _append(lens, new, T, Hq, Hkv, d, dtype, rot, interleaved, *, heads_first=False, fused=True, q_start=True, seed=0,
            tail_rows=0, with_q=True, in_place=False):
    P = Paged(lens, T, Hkv, d, dtype, seed=seed, heads_first=heads_first, fill=False)
    g = torch.Generator().manual_seed(seed + 1)
    N = sum(new) + tail_rows
    qkv = torch.randn(N, Hq + 2 * Hkv, d, generator=g).to(dtype).to(DEV)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q0, k0, v0 = (x.double().cpu() for x in (q, k, v))
    cs = cos_sin(max(lens) + 3, rot).to(DEV) if rot else None
    q_out = q if in_place else torch.full((N, Hq, d), 7.0, dtype=dtype, device=DEV)
    k_before, v_before = P.k.clone(), P.v.clone()
    got = E.paged_append(k, v, P.k, P.v, P.table, P.seq_len, q=q if with_q else None, q_out=q_out if with_q else None,
                         cos_sin=cs, interleaved=interleaved, q_start=starts(new) if q_start else None,
                         status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    r = 0
    # the rotated values: two products and a sum in float32, one rounding to the type
    tol = lambda a, b: 1.01 * half_step(dtype) * b.abs() + 3 * 2.0 ** -24 * a  # noqa: E731
    for b, n in enumerate(new):
        pos = torch.arange(lens[b] - n, lens[b])
        kq = k0[r:r + n], q0[r:r + n]
        if rot:
            c = cs.cpu()[pos]
            want_k, want_q = rotate(kq[0], c, interleaved), rotate(kq[1], c, interleaved)
        else:
            want_k, want_q = kq
        if n:
            pg, row = P.at(b, pos)
            at = lambda x: x[pg, row].double().cpu()  # noqa: E731
            size = kq[0].abs().amax() * 2
            assert torch.all((at(P.k) - want_k).abs() <= tol(size, want_k)), f"keys of {b}"
            assert torch.equal(at(P.v), v0[r:r + n]), f"values of {b}"
            if with_q and Hq:
                w = got[r:r + n].double().cpu()
                assert torch.all((w - want_q).abs() <= tol(kq[1].abs().amax() * 2, want_q)), f"queries of {b}"
            k_before[pg, row], v_before[pg, row] = P.k[pg, row], P.v[pg, row]
        r += n
    same = lambda a, b: torch.equal(a.nan_to_num(3.0), b.nan_to_num(3.0))  # noqa: E731
    assert same(P.k, k_before) and same(P.v, v_before), "other rows of the pool"
    if with_q and tail_rows and not in_place:
        assert torch.all(got[r:] == 7.0), "rows behind the last sequence"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 64, True), (64, 16, False),
                                               (128, 0, False), (64, 48, False), (128, 112, True)])
def test_append_ragged_chunks(dtype, d, rot, interleaved):
    _append([70, 3, 40, 1, 129], [33, 3, 0, 1, 129], 16, 6, 2, d, dtype, rot, interleaved, tail_rows=3, seed=d + rot)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 7, 64])
def test_append_one_token_each(dtype, T):
    lens = [1, 2, 65, 1000, 64, 7, 8, 300]
    _append(lens, [1] * 8, T, 10, 2, 128, dtype, 128, False, q_start=False, heads_first=T == 7)


def test_append_many_sequences_and_odd_head_counts():
    _append([1 + (7 * i) % 50 for i in range(700)], [1] * 700, 8, 3, 1, 64, BF, 64, False, q_start=True)
    _append([20 + i % 9 for i in range(300)], [i % 4 for i in range(300)], 24, 7, 7, 128, BF, 32, True)


def test_append_keys_and_values_alone_and_queries_in_place():
    _append([90, 31], [40, 31], 16, 4, 4, 128, BF, 128, False, with_q=False)
    _append([90, 31], [40, 31], 16, 8, 2, 128, BF, 128, False, fused=False, in_place=True)
    _append([90, 31], [40, 31], 16, 8, 2, 64, F32, 64, True, fused=False, in_place=True)


def test_append_bad_page_and_position():
    P = Paged([20, 20, 20], 8, 2, 64, BF, fill=False)
    table = P.table.clone()
    table[1, 2] = P.n_pages                              # tokens 16 .. 19 of sequence 1
    k, v, q = (torch.ones(12, h, 64, dtype=BF, device=DEV) for h in (2, 2, 4))
    q_out = torch.zeros(12, 4, 64, dtype=BF, device=DEV)
    E.paged_append(k, v, P.k, P.v, table, P.seq_len, q=q, q_out=q_out, q_start=starts([4, 4, 4]), status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.ERR_PAGE
    assert int(torch.isfinite(P.k).sum()) == 8 * 2 * 64 and bool(torch.all(q_out == 1))
    # positions past the page table, before zero, and past the rotation's table
    for lens, cs in (([1000, 20, 20], None), ([3, 20, 20], None), ([20, 20, 20], cos_sin(18, 64).to(DEV))):
        P.k.fill_(math.nan)
        P.status.zero_()
        q_out.zero_()
        seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
        E.paged_append(k, v, P.k, P.v, P.table, seq, q=q, q_out=q_out, q_start=starts([4, 4, 4]), cos_sin=cs,
                       status=P.status)
        torch.cuda.synchronize()
        rows = {1000: 8, 3: 11, 20: 6}[lens[0]]
        assert P.status.item() == E.ERR_INVALID_ARG
        assert int(torch.isfinite(P.k).sum()) == rows * 2 * 64
        assert int((q_out != 0).any(2).any(1).sum()) == rows


# ----------------------------------------------------------------- one new token --
def _decode(lens, T, Hq, Hkv, d, dtype, *, seed=0, heads_first=False, cap=0.0, window=0, alibi=False, first=None,
            prefix=None, q_scale=1.0, fused=False):
    P = Paged(lens, T, Hkv, d, dtype, seed=seed, heads_first=heads_first)
    g = torch.Generator().manual_seed(seed + 1)
    B = len(lens)
    q = (torch.randn(B, Hq + (2 if fused else 0), d, generator=g) * q_scale).to(dtype).to(DEV)[:, :Hq]
    slopes = 2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq) if alibi else None
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out, lse = E.paged_attn_decode(q, P.k, P.v, P.table, P.seq_len, d ** -0.5, softcap=cap, window=window,
                                   slopes=None if slopes is None else slopes.to(DEV), first_tok=i32(first),
                                   prefix_len=i32(prefix), status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    for b, n in enumerate(lens):
        ref = attend(q[b:b + 1].double().cpu(), P.K[b], P.V[b], [n - 1], d ** -0.5, dtype=dtype, cap=cap, window=window,
                     slopes=slopes, first=None if first is None else [first[b]],
                     prefix=0 if prefix is None else prefix[b])
        check_rows(f"sequence {b} of {n}", out[b:b + 1], lse[b:b + 1], ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 128), (16, 2, 64), (5, 5, 128), (20, 4, 64), (32, 2, 128), (24, 1, 64),
                                      (128, 1, 128)])
def test_decode_head_layouts_and_lengths(dtype, Hq, Hkv, d):
    _decode([0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 500, 129], 16, Hq, Hkv, d, dtype, seed=Hq + d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 5, 24, 64, 100, 256])
def test_decode_page_sizes(dtype, T):
    _decode([777, 3, 64, 0, 1300], T, 12, 4, 128, dtype, seed=T, heads_first=T in (5, 64))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_one_long_sequence_is_split_and_joined(dtype):
    _decode([60013], 16, 16, 2, 128, dtype, seed=5)
    _decode([9001, 1, 17], 32, 3, 3, 64, dtype, seed=6)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_many_sequences_with_empty_ones(dtype):
    lens = [(i * 37) % 211 if i % 3 else 0 for i in range(400)]
    _decode(lens, 16, 4, 2, 64, dtype, seed=7)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(cap=5.0, q_scale=6.0), dict(alibi=True), dict(window=1), dict(window=100),
                                dict(window=64, prefix=True), dict(window=200, prefix=True, alibi=True, cap=30.0),
                                dict(first=True), dict(first=True, prefix=True, window=50)])
def test_decode_masks_and_modifiers(dtype, kw):
    lens = [1, 64, 65, 300, 1025, 700, 130]
    kw = dict(kw)
    if kw.pop("prefix", None):
        kw["prefix"] = [4, 70, 1, 64, 129, 700, 0]
    if kw.pop("first", None):
        kw["first"] = [0, 63, 65, 100, 3, 699, 64]       # the third sees nothing
    _decode(lens, 16, 8, 2, 128, dtype, seed=9, **kw)


def test_decode_large_scores_and_strided_queries():
    _decode([300, 70], 16, 8, 2, 128, F32, q_scale=200.0, seed=3)
    _decode([300, 70], 16, 8, 2, 64, BF, fused=True, seed=4)


def test_decode_pages_nobody_sees_are_not_read_and_bad_ones_are_skipped():
    P = Paged([500, 500], 16, 2, 128, BF, seed=2)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    full = E.paged_attn_decode(q, P.k, P.v, P.table, P.seq_len, 0.1, window=70)
    table = P.table.clone()
    table[:, :(500 - 70) // 16] = -1                     # pages behind the window were given back
    P.k[P.table[:, :(500 - 70) // 16].flatten().long()] = math.nan
    P.v[P.table[:, :(500 - 70) // 16].flatten().long()] = math.nan
    got = E.paged_attn_decode(q, P.k, P.v, table, P.seq_len, 0.1, window=70, status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK and all(torch.equal(a, b) for a, b in zip(full, got))
    # a bad page among the seen ones: flagged, its tokens left out
    table[0, 30] = P.n_pages + 5
    out, lse = E.paged_attn_decode(q, P.k, P.v, table, P.seq_len, 0.1, window=70, status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.ERR_PAGE and bool(torch.isfinite(out).all())
    assert torch.equal(out[1], full[0][1])
    keep = torch.tensor([t for t in range(430, 500) if t // 16 != 30])
    ref = attend(q[:1].double().cpu(), P.K[0][keep], P.V[0][keep], [len(keep) - 1], 0.1, dtype=BF)
    check_rows("without the bad page", out[:1], lse[:1], ref)


def test_decode_length_past_the_page_table_is_cut_and_flagged():
    P = Paged([100], 16, 1, 64, F32, room=[112])
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(1)).to(DEV)
    table = P.table[:, :6].contiguous()                  # 96 tokens
    out, lse = E.paged_attn_decode(q, P.k, P.v, table, P.seq_len, 0.1, status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.ERR_INVALID_ARG
    check_rows("cut", out, lse, attend(q.double().cpu(), P.K[0][:96], P.V[0][:96], [95], 0.1, dtype=F32))


def test_offsets_past_32_bits():
    # a pool of 2^31 + values for the keys: the sequence's pages lie at its far end
    T, Hkv, d = 64, 8, 128
    n_pages = (1 << 31) // (T * Hkv * d) + 40
    k, v = (torch.empty(n_pages, T, Hkv, d, dtype=BF, device=DEV) for _ in range(2))
    g = torch.Generator().manual_seed(3)
    lens, new = [130, 70], [130, 70]
    table = torch.tensor([[n_pages - 1, n_pages - 5, n_pages - 2], [n_pages - 7, 0, -1]], dtype=torch.int32, device=DEV)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    x = torch.randn(200, 32, d, generator=g).to(BF).to(DEV)
    q, kk, vv = x[:, :16], x[:, 16:24], x[:, 24:]
    E.paged_append(kk, vv, k, v, table, seq, q_start=starts(new))
    out, lse = E.paged_attn_prefill(q, starts(new), k, v, table, seq, d ** -0.5)
    last = torch.tensor([129, 199], device=DEV)
    o1, l1 = E.paged_attn_decode(q[last].contiguous(), k, v, table, seq, d ** -0.5)
    torch.cuda.synchronize()
    c = x.double().cpu()
    for r0, n in ((0, 130), (130, 70)):
        s = slice(r0, r0 + n)
        ref = attend(c[s, :16], c[s, 16:24], c[s, 24:], range(n), d ** -0.5, dtype=BF)
        check_rows("prompt", out[s], lse[s], ref)
        i = 0 if r0 == 0 else 1
        check_rows("token", o1[i:i + 1], l1[i:i + 1], tuple(y[-1:] for y in ref))


# --------------------------------------------------------------- many new tokens --
def _prefill(lens, new, T, Hq, Hkv, d, dtype, *, seed=0, heads_first=False, cap=0.0, window=0, alibi=False, docs=0,
             prefix=None, first=None, q_scale=1.0, tail_rows=0, fused=False, heads=None):
    P = Paged(lens, T, Hkv, d, dtype, seed=seed, heads_first=heads_first)
    g = torch.Generator().manual_seed(seed + 1)
    N = sum(new) + tail_rows
    q = (torch.randn(N, Hq + (1 if fused else 0), d, generator=g) * q_scale).to(dtype).to(DEV)[:, :Hq]
    slopes = 2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq) if alibi else None
    if docs:
        first = [int(doc_starts(lens[b], docs, seed + b)[lens[b] - n + i]) for b, n in enumerate(new) for i in range(n)]
    if first is not None:
        first = list(first) + [0] * (N - len(first))
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out = torch.full((N, Hq, d), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((N, Hq), 7.0, device=DEV)
    E.paged_attn_prefill(q, starts(new), P.k, P.v, P.table, P.seq_len, d ** -0.5, softcap=cap, window=window,
                         slopes=None if slopes is None else slopes.to(DEV), first_tok=i32(first),
                         prefix_len=i32(prefix), out=out, lse=lse, status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    r = 0
    for b, n in enumerate(new):
        if n:
            s = slice(r, r + n)
            ref = attend(q[s].double().cpu(), P.K[b], P.V[b], range(lens[b] - n, lens[b]), d ** -0.5, dtype=dtype,
                         cap=cap, window=window, slopes=slopes, first=None if first is None else first[s],
                         prefix=0 if prefix is None else prefix[b])
            check_rows(f"sequence {b}: {n} of {lens[b]}", out[s], lse[s], ref)
        r += n
    assert bool(torch.all(out[r:] == 7.0)) and bool(torch.all(lse[r:] == 7.0)), "rows behind the last sequence"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 128), (8, 2, 64), (3, 3, 128), (10, 2, 64), (16, 1, 128), (36, 1, 64),
                                      (128, 1, 128)])
def test_prefill_head_layouts_ragged(dtype, Hq, Hkv, d):
    new = [0, 1, 2, 17, 64, 65, 130]
    _prefill([9, 1, 50, 17, 64, 300, 131], new, 16, Hq, Hkv, d, dtype, seed=Hq + d, tail_rows=5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 5, 24, 64, 100, 256])
def test_prefill_page_sizes(dtype, T):
    _prefill([333, 90], [200, 90], T, 6, 2, 128, dtype, seed=T, heads_first=T in (5, 64))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_long_prompt_and_chunk(dtype):
    _prefill([1111], [1111], 16, 4, 2, 128, dtype, seed=11)
    _prefill([5000, 4100], [77, 3], 32, 8, 2, 64, dtype, seed=12, fused=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_drafted_tokens(dtype):
    _prefill([3000, 2999, 40, 4, 1500], [4, 4, 4, 4, 2], 16, 16, 2, 128, dtype, seed=13)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(cap=5.0, q_scale=6.0), dict(alibi=True), dict(window=1), dict(window=100),
                                dict(window=64, prefix=True), dict(window=150, prefix=True, alibi=True, cap=30.0),
                                dict(docs=20), dict(docs=90, alibi=True), dict(prefix=True),
                                dict(docs=40, prefix=True, window=33)])
def test_prefill_masks_and_modifiers(dtype, kw):
    kw = dict(kw)
    if kw.pop("prefix", None):
        kw["prefix"] = [70, 333, 128, 1, 0]
    _prefill([70, 333, 260, 200, 500], [70, 333, 9, 64, 130], 16, 8, 2, 128, dtype, seed=21, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_rows_that_see_nothing(dtype):
    # document starts behind the row itself leave it empty; a whole tile of empty rows too
    n = 300
    first = [i + 1 if (i % 3 == 0 or 64 <= i < 200) else max(0, i - 5) for i in range(n)]
    _prefill([n, 20], [n, 20], 16, 4, 1, 64, dtype, seed=31, first=first + [0] * 20)


def test_prefill_large_scores():
    _prefill([300], [300], 16, 4, 2, 128, F32, q_scale=100.0, seed=33)
    _prefill([300], [300], 16, 4, 2, 128, BF, q_scale=30.0, seed=34)


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_scales_of_zero_and_below(scale):
    P = Paged([150], 16, 1, 64, BF, seed=36)
    q = torch.randn(90, 3, 64, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    for cap in (0.0, 2.0):
        out, lse = E.paged_attn_prefill(q, starts([90]), P.k, P.v, P.table, P.seq_len, scale, softcap=cap)
        ref = attend(q.double().cpu(), P.K[0], P.V[0], range(60, 150), scale, dtype=BF, cap=cap)
        check_rows("prompt", out, lse, ref)
        out, lse = E.paged_attn_decode(q[-1:], P.k, P.v, P.table, P.seq_len, scale, softcap=cap)
        check_rows("token", out, lse, tuple(x[-1:] for x in ref))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(window=200), dict(cap=5.0, q_scale=6.0, alibi=True), dict(docs=200),
                                dict(prefix=True, alibi=True), dict(empty=True)])
def test_prefill_short_runs_of_rows_beside_long_ones(d, kw):
    # a few new tokens each over caches of one tile, two and many, between prompts of several row
    # tiles: row tiles of one query tile and of two follow one another on a CTA
    kw = dict(kw)
    new = [(1, 4, 3, 150, 4, 0, 2, 33, 4, 4, 60)[i % 11] for i in range(37)]
    lens = [n + (0, 700, 120, 9, 128, 5, 1000, 256, 129, 2000, 380)[(i * 5) % 11] for i, n in enumerate(new)]
    if kw.pop("prefix", None):
        kw["prefix"] = [(0, 300, 5)[i % 3] for i in range(37)]
    if kw.pop("empty", None):
        # half of every sequence's rows see nothing, one in three only their last tokens
        kw["first"] = [p + 1 if p % 2 else (max(0, p - 40) if p % 3 == 0 else 0)
                       for n, m in zip(lens, new) for p in range(n - m, n)]
    _prefill(lens, new, 16, 8, 2, d, BF, seed=51, tail_rows=2, **kw)


def test_prefill_many_sequences():
    new = [i % 4 for i in range(300)]
    _prefill([n + (11 * i) % 40 for i, n in enumerate(new)], new, 8, 4, 2, 64, BF, seed=35)


def test_prefill_bad_pages_and_lengths():
    P = Paged([200, 200], 16, 2, 128, BF, seed=2)
    q = torch.randn(80, 4, 128, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    qs = starts([40, 40])
    good = E.paged_attn_prefill(q, qs, P.k, P.v, P.table, P.seq_len, 0.1, window=30)
    table = P.table.clone()
    table[:, :(160 - 30) // 16] = -1                     # given back: nobody sees them
    got = E.paged_attn_prefill(q, qs, P.k, P.v, table, P.seq_len, 0.1, window=30, status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK and all(torch.equal(a, b) for a, b in zip(good, got))
    table[0, 11] = -7                                    # tokens 176 .. 191
    out, lse = E.paged_attn_prefill(q, qs, P.k, P.v, table, P.seq_len, 0.1, window=30, status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.ERR_PAGE and bool(torch.isfinite(out).all())
    assert torch.equal(out[40:], good[0][40:]) and torch.equal(out[:16], good[0][:16])
    # a sequence shorter than its new rows: the rows before its start see nothing
    P.status.zero_()
    seq = torch.tensor([200, 30], dtype=torch.int32, device=DEV)
    out, lse = E.paged_attn_prefill(q, qs, P.k, P.v, P.table, seq, 0.1, status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.ERR_INVALID_ARG
    assert bool(torch.isneginf(lse[40:50]).all()) and not out[40:50].any()
    ref = attend(q[50:].double().cpu(), P.K[1][:30], P.V[1][:30], range(30), 0.1, dtype=BF)
    check_rows("the rest", out[50:], lse[50:], ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("qs,code", [([0, 0, 0, 0], E.OK), ([5, 5, 5, 5], E.OK), ([0, 60, 20, 80], E.ERR_INVALID_ARG),
                                     ([0, 70, -5, 70], E.ERR_INVALID_ARG), ([100, 100, 90, 100], E.OK)])
def test_prefill_without_rows_or_with_descending_starts(dtype, qs, code):
    # (entries past the 80 rows are cut to 80: the last one has no row)
    P = Paged([200, 100, 90], 16, 2, 64, dtype, seed=3)
    q = torch.randn(80, 4, 64, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    out, lse = torch.full_like(q, 7.0), torch.full((80, 4), 7.0, device=DEV)
    E.paged_attn_prefill(q, torch.tensor(qs, dtype=torch.int32, device=DEV), P.k, P.v, P.table, P.seq_len, 0.1,
                         out=out, lse=lse, status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == code
    assert bool(torch.all(out == 7.0)) and bool(torch.all(lse == 7.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_results_at_any_16_byte_boundary_and_a_dirty_workspace(dtype, d):
    P = Paged([1500, 40, 700], 16, 2, d, dtype, seed=5)
    g = torch.Generator().manual_seed(1)
    c, off = 16 // dtype.itemsize, 8 // dtype.itemsize * 2

    def shifted(*shape):                                 # 16 bytes past a 256-byte boundary
        n = torch.Size(shape).numel()
        return torch.empty(n + c, dtype=dtype, device=DEV)[off:off + n].view(shape)

    q = shifted(150, 8, d).copy_(torch.randn(150, 8, d, generator=g))
    qs = starts([100, 5, 45])
    want = E.paged_attn_prefill(q, qs, P.k, P.v, P.table, P.seq_len, 0.1)
    last = [99, 104, 149]
    one = E.paged_attn_decode(q[last].contiguous(), P.k, P.v, P.table, P.seq_len, 0.1)
    for n, call, ref in ((E.paged_prefill_workspace_bytes(150, 3, 8, 2, d), E.paged_attn_prefill, want),
                         (E.paged_decode_workspace_bytes(8, 2, d), E.paged_attn_decode, one)):
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        out = shifted(*ref[0].shape)
        x = (q, qs) if call is E.paged_attn_prefill else (q[last].contiguous(),)
        got = call(*x, P.k, P.v, P.table, P.seq_len, 0.1, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert got[0] is out and torch.equal(out, ref[0]) and torch.equal(got[1], ref[1])


# ---------------------------------------------------------------------- together --
def test_a_request_from_prompt_to_tokens_in_one_graph():
    """Two requests: prompts appended and attended, then tokens one by one, the token step
    captured once and replayed as the sequences grow; every result against dense attention."""
    T, Hq, Hkv, d, steps = 16, 8, 2, 128, 5
    prompt, scale = [75, 130], d ** -0.5
    P = Paged([0, 0], T, Hkv, d, BF, room=[n + steps for n in prompt])
    cs = cos_sin(200, d).to(DEV)
    g = torch.Generator().manual_seed(1)
    data = [torch.randn(n + steps, Hq + 2 * Hkv, d, generator=g).to(BF) for n in prompt]

    def split(x):
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def check(b, pos, q, out, lse):
        # the pages hold the rotated keys and the values as they came; attention is over them
        end = max(pos) + 1
        pg, row = P.at(b, torch.arange(end))
        K, V = P.k[pg, row].double().cpu(), P.v[pg, row].double().cpu()
        want = rotate(data[b][:end, Hq:Hq + Hkv], cs.cpu()[:end], False)
        assert torch.all((K - want).abs() <= 1.01 * half_step(BF) * want.abs() + 2.0 ** -20)
        assert torch.equal(V, data[b][:end, Hq + Hkv:].double())
        want = rotate(data[b][pos[0]:end, :Hq], cs.cpu()[pos[0]:end], False)
        assert torch.all((q.double().cpu() - want).abs() <= 1.01 * half_step(BF) * want.abs() + 2.0 ** -20)
        check_rows(f"request {b} at {pos[0]}", out, lse, attend(q.double().cpu(), K, V, pos, scale, dtype=BF))

    qs = starts(prompt)
    P.seq_len.copy_(torch.tensor(prompt, dtype=torch.int32))
    q, k, v = split(torch.cat([x[:n] for x, n in zip(data, prompt)]).to(DEV))
    qr = E.paged_append(k, v, P.k, P.v, P.table, P.seq_len, q=q, cos_sin=cs, q_start=qs, status=P.status)
    out, lse = E.paged_attn_prefill(qr, qs, P.k, P.v, P.table, P.seq_len, scale, status=P.status)
    torch.cuda.synchronize()
    for b, n in enumerate(prompt):
        s = slice(int(qs[b]), int(qs[b]) + n)
        check(b, range(n), qr[s], out[s], lse[s])

    x = torch.zeros(2, Hq + 2 * Hkv, d, dtype=BF, device=DEV)
    q, k, v = split(x)
    qr = torch.empty(2, Hq, d, dtype=BF, device=DEV)
    out, lse = torch.empty_like(qr), torch.empty(2, Hq, device=DEV)
    ws = torch.empty(E.paged_decode_workspace_bytes(Hq, Hkv, d), dtype=torch.uint8, device=DEV)

    def step():
        P.seq_len.add_(1)
        E.paged_append(k, v, P.k, P.v, P.table, P.seq_len, q=q, q_out=qr, cos_sin=cs, status=P.status)
        E.paged_attn_decode(qr, P.k, P.v, P.table, P.seq_len, scale, out=out, lse=lse, workspace=ws, status=P.status)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        x.copy_(torch.stack([d_[n] for d_, n in zip(data, prompt)]))
        step()                                           # a first token, eagerly, on another stream
    side.synchronize()
    for b, n in enumerate(prompt):
        check(b, [n], qr[b:b + 1], out[b:b + 1], lse[b:b + 1])
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(1, steps):
        x.copy_(torch.stack([d_[n + i] for d_, n in zip(data, prompt)]))
        ws.fill_(255)                                    # nothing is kept in the workspace
        graph.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(prompt):
            check(b, [n + i], qr[b:b + 1], out[b:b + 1], lse[b:b + 1])
    assert P.status.item() == E.OK


@pytest.mark.parametrize("dtype", [BF, F32])
def test_results_do_not_change_between_calls(dtype):
    P = Paged([4000, 30, 900], 16, 2, 128, dtype, seed=4)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(3, 16, 128, generator=g).to(dtype).to(DEV)
    qq = torch.randn(120, 16, 128, generator=g).to(dtype).to(DEV)
    first = None
    for _ in range(3):
        a = E.paged_attn_decode(q, P.k, P.v, P.table, P.seq_len, 0.1)
        b = E.paged_attn_prefill(qq, starts([100, 5, 15]), P.k, P.v, P.table, P.seq_len, 0.1)
        torch.cuda.synchronize()
        first = first or (*a, *b)
        assert all(torch.equal(x, y) for x, y in zip(first, (*a, *b)))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_captured_prompt_call_serves_other_lengths(dtype):
    # captured once over 64 rows, replayed with other rows, lengths and documents
    P = Paged([900, 300, 40], 16, 2, 64, dtype, seed=8)
    q = torch.randn(64, 8, 64, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    qs, first = starts([40, 20, 4]), torch.zeros(64, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(64, 8, device=DEV)
    ws = torch.empty(E.paged_prefill_workspace_bytes(64, 3, 8, 2, 64), dtype=torch.uint8, device=DEV)

    def call():
        E.paged_attn_prefill(q, qs, P.k, P.v, P.table, P.seq_len, 0.1, first_tok=first, out=out, lse=lse, workspace=ws,
                             status=P.status)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, new, f in (([900, 300, 40], [40, 20, 4], 0), ([700, 17, 0], [4, 4, 0], 0), ([64, 1, 1], [62, 1, 1], 10)):
        qs.copy_(starts(new))
        P.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        first.fill_(f)
        out.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        r = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            if m:
                ref = attend(q[r:r + m].double().cpu(), P.K[b][:n], P.V[b][:n], range(n - m, n), 0.1, dtype=dtype,
                             first=[f] * m)
                check_rows(f"{m} of {n}", out[r:r + m], lse[r:r + m], ref)
            r += m
        assert bool(torch.all(out[r:] == 7.0))
    assert P.status.item() == E.OK


def test_given_stream_and_two_streams_at_once():
    P = Paged([3000, 64], 16, 2, 128, BF, seed=6)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    want = E.paged_attn_decode(q, P.k, P.v, P.table, P.seq_len, 0.1)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    got = [E.paged_attn_decode(q, P.k, P.v, P.table, P.seq_len, 0.1, stream=s[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    for o, z in got:
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])


def test_shared_pages_are_read_by_both_sequences():
    P = Paged([64, 64], 16, 2, 64, BF, seed=8)
    table = P.table.clone()
    table[1, :2] = table[0, :2]                          # a shared beginning
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    out, lse = E.paged_attn_decode(q, P.k, P.v, table, P.seq_len, 0.125)
    torch.cuda.synchronize()
    K, V = torch.cat([P.K[0][:32], P.K[1][32:]]), torch.cat([P.V[0][:32], P.V[1][32:]])
    check_rows("second", out[1:], lse[1:], attend(q[1:].double().cpu(), K, V, [63], 0.125, dtype=BF))


# ----------------------------------------------------------------------- refusals --
def _args(**kw):
    P = Paged([20, 9], 8, 2, 64, BF)
    a = dict(q=torch.zeros(2, 4, 64, dtype=BF, device=DEV), k_pages=P.k, v_pages=P.v, page_table=P.table,
             seq_len=P.seq_len, scale=0.1)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(q=torch.zeros(3, 4, 64, dtype=BF)), E.ERR_INVALID_ARG),
    (dict(q=torch.zeros(2, 3, 64, dtype=BF)), E.ERR_UNSUPPORTED),                 # 3 heads over 2
    (dict(q=torch.zeros(2, 4, 32, dtype=BF)), E.ERR_INVALID_ARG),
    (dict(q=torch.zeros(2, 4, 64)), E.ERR_INVALID_ARG),
    (dict(scale=math.nan), E.ERR_INVALID_ARG), (dict(softcap=-1.0), E.ERR_INVALID_ARG),
    (dict(softcap=math.inf), E.ERR_INVALID_ARG), (dict(window=-1), E.ERR_INVALID_ARG),
    (dict(slopes=torch.zeros(3)), E.ERR_INVALID_ARG), (dict(slopes=torch.zeros(4, dtype=BF)), E.ERR_INVALID_ARG),
    (dict(first_tok=torch.zeros(3, dtype=torch.int32)), E.ERR_INVALID_ARG),
    (dict(prefix_len=torch.zeros(2, dtype=torch.int64)), E.ERR_INVALID_ARG),
    (dict(seq_len=torch.zeros(3, dtype=torch.int32)), E.ERR_INVALID_ARG),
    (dict(page_table=torch.zeros(2, 3, dtype=torch.int64)), E.ERR_INVALID_ARG),
    (dict(out=torch.zeros(2, 4, 64)), E.ERR_INVALID_ARG), (dict(lse=torch.zeros(2, 4, dtype=BF)), E.ERR_INVALID_ARG),
    (dict(workspace=torch.zeros(64, dtype=torch.uint8)), E.ERR_INVALID_ARG),
])
def test_decode_refusals(kw, code):
    kw = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    with pytest.raises(E.EchoError) as e:
        E.paged_attn_decode(**_args(**kw))
    assert e.value.code == code


def test_layout_refusals():
    def z(*shape, dtype=BF):
        return torch.zeros(*shape, dtype=dtype, device=DEV)

    for k, v, code in [
        (z(4, 8, 2, 64), z(4, 8, 2, 64, dtype=F32), E.ERR_INVALID_ARG),
        (z(4, 8, 2, 64, dtype=torch.float16), z(4, 8, 2, 64, dtype=torch.float16), E.ERR_UNSUPPORTED),
        (z(4, 8, 2, 96), z(4, 8, 2, 96), E.ERR_UNSUPPORTED),
        (z(4, 2, 8, 64).transpose(1, 2), z(4, 8, 2, 64), E.ERR_INVALID_ARG),
        (z(4, 8, 2, 68)[..., :64], z(4, 8, 2, 68)[..., :64], E.ERR_INVALID_ARG),       # rows not 16 bytes apart
        (z(4, 8, 2, 72)[..., 4:68], z(4, 8, 2, 72)[..., 4:68], E.ERR_INVALID_ARG),     # rows not 16-byte aligned
        (z(4, 8, 2, 64).cpu(), z(4, 8, 2, 64).cpu(), E.ERR_INVALID_ARG),
    ]:
        q = torch.zeros(2, 4, k.shape[3], dtype=k.dtype, device=DEV)
        with pytest.raises(E.EchoError) as e:
            E.paged_attn_decode(**_args(q=q, k_pages=k, v_pages=v))
        assert e.value.code == code


def test_append_and_prefill_refusals():
    a = _args()
    kv = torch.zeros(2, 2, 64, dtype=BF, device=DEV)
    pages = (a["k_pages"], a["v_pages"], a["page_table"], a["seq_len"])
    i32 = dict(dtype=torch.int32, device=DEV)
    for bad, code in [
        (dict(cos_sin=torch.zeros(32, 24, device=DEV)), E.ERR_UNSUPPORTED),
        (dict(cos_sin=torch.zeros(32, 128, device=DEV)), E.ERR_UNSUPPORTED),
        (dict(cos_sin=torch.zeros(32, 64, dtype=BF, device=DEV)), E.ERR_INVALID_ARG),
        (dict(q_start=torch.zeros(2, **i32)), E.ERR_INVALID_ARG),
        (dict(q_out=a["q"]), E.ERR_INVALID_ARG),
        (dict(q=a["q"].transpose(0, 1)), E.ERR_INVALID_ARG),
    ]:
        with pytest.raises(E.EchoError) as e:
            E.paged_append(kv, kv, *pages, **bad)
        assert e.value.code == code, bad
    with pytest.raises(E.EchoError):
        E.paged_append(kv[:1], kv[:1], *pages)                  # one row for two sequences
    with pytest.raises(E.EchoError):
        E.paged_append(kv, kv[:1], *pages)
    for bad in (dict(q_start=None), dict(q_start=torch.zeros(2, **i32)), dict(q_start=torch.zeros(3, device=DEV))):
        with pytest.raises(E.EchoError) as e:
            E.paged_attn_prefill(a["q"], bad["q_start"], *pages, 0.1)
        assert e.value.code == E.ERR_INVALID_ARG
