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


# -------------------------------------------------------- a stream of the call's own --
def _call_beside_pending_work(call, shapes):
    """call() with default buffers on a stream of its own while the current stream still has work on blocks
    of `shapes` (shape, type) that are already free again: writes to some of them and a read of
    others.  Neither may meet the call's buffers."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [(torch.empty(s, dtype=t, device=DEV), torch.ones(s, dtype=t, device=DEV)) for s, t in shapes]
    copies = [torch.empty(s, dtype=t, device=DEV) for s, t in shapes]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                       # some 50 ms
    for (x, y), c in zip(held, copies):
        x.fill_(3)
        c.copy_(y)
    del held, x, y
    got = call()
    torch.cuda.synchronize()
    assert all(bool((c == 1).all()) for c in copies), "a pending read of a freed block"
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
def test_default_buffers_on_a_given_stream_with_work_pending_on_the_current_one(dtype):
    Hq, Hkv, d, T = 16, 2, 128, 16
    P = Paged([20000, 300], T, Hkv, d, dtype, seed=3)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, Hq, d, generator=g).to(dtype).to(DEV)
    qq = torch.randn(40, Hq, d, generator=g).to(dtype).to(DEV)
    kv = torch.randn(2, Hkv, d, generator=g).to(dtype).to(DEV)
    qs = torch.tensor([0, 30, 40], dtype=torch.int32, device=DEV)
    cs = torch.rand(20000, d, generator=g).to(DEV)
    side = torch.cuda.Stream()
    u8 = torch.uint8
    for call, shapes in (
            (lambda s: E.paged_attn_decode(q, P.k, P.v, P.table, P.seq_len, 0.1, stream=s),
             [((2, Hq, d), dtype), ((2, Hq), F32), ((E.paged_decode_workspace_bytes(Hq, Hkv, d),), u8)]),
            (lambda s: E.paged_attn_prefill(qq, qs, P.k, P.v, P.table, P.seq_len, 0.1, stream=s),
             [((40, Hq, d), dtype), ((40, Hq), F32), ((E.paged_prefill_workspace_bytes(40, 2, Hq, Hkv, d),), u8)]),
            (lambda s: [E.paged_append(kv, kv, P.k, P.v, P.table, P.seq_len, q=q, cos_sin=cs, stream=s)],
             [((2, Hq, d), dtype)])):
        want = [x.clone() for x in call(None)]
        got = _call_beside_pending_work(lambda: call(side), shapes)  # noqa: B023
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------ tokens that no row of a call sees --
def _rows_first(kind, lens, new):
    """First tokens of every row: rows of padding see nothing (their first token lies behind
    them), the others see their document."""
    first = []
    for n, m in zip(lens, new):
        for i, p in enumerate(range(n - m, n)):
            if kind == "tail":                           # the last third of each sequence is padding
                first.append(0x7fffffff if i >= m - m // 3 else 0)
            elif kind == "documents":                    # documents of 23 tokens, padded to 32
                first.append(n if p % 32 >= 23 else p // 32 * 32)
            elif kind == "head":                         # the first rows are padding
                first.append(p + 1 if i < m // 2 else max(0, p - 3))
            else:                                        # a few rows here and there see something
                first.append(max(0, p - 40) if i % 17 == 3 else p + 1 + i % 5)
    return first


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d,T", [(8, 2, 128, 16), (3, 3, 64, 5), (16, 1, 64, 8)])
@pytest.mark.parametrize("kind", ["tail", "documents", "head", "sparse"])
@pytest.mark.parametrize("kw", [dict(), dict(window=9), dict(prefix=(7, 0, 70)), dict(window=30, prefix=(0, 40, 1))])
@pytest.mark.parametrize("lens,new", [([150, 9, 300], [150, 6, 120]), ([500, 40, 700], [7, 6, 8])])
def test_prefill_tokens_that_no_row_sees_may_hold_anything(dtype, Hq, Hkv, d, T, kind, kw, lens, new):
    """Padding tokens (below seq_len, but outside every row's sight) are NaN in the cache, and pages
    that hold nothing else are not in the table: not an error, and no row's result."""
    P = Paged(lens, T, Hkv, d, dtype, seed=11)
    first, prefix, window = _rows_first(kind, lens, new), kw.get("prefix"), kw.get("window", 0)
    table, r = P.table.clone(), 0
    for b, (n, m) in enumerate(zip(lens, new)):
        t, p = torch.arange(n), torch.arange(n - m, n)[:, None]
        see = (t <= p) & (t > p - window if window else t >= 0)
        if prefix:
            see = see | (t < prefix[b])
        see = (see & (t >= torch.tensor(first[r:r + m])[:, None])).any(0)
        pg, row = P.at(b, t[~see])
        P.k[pg, row], P.v[pg, row] = float("nan"), float("nan")
        for i in range(-(-n // T)):
            if not see[i * T:(i + 1) * T].any():
                table[b, i] = -1
        r += m
    q = torch.randn(r, Hq, d, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    qs = i32([0, *torch.tensor(new).cumsum(0).tolist()])
    out, lse = E.paged_attn_prefill(q, qs, P.k, P.v, table, P.seq_len, 0.1, window=window, first_tok=i32(first),
                                    prefix_len=i32(prefix), status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    r = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        s = slice(r, r + m)
        ref = attend(q[s].double().cpu(), P.K[b], P.V[b], range(n - m, n), 0.1, dtype=dtype, window=window,
                     first=first[s], prefix=prefix[b] if prefix else 0)
        check_rows(f"sequence {b}", out[s], lse[s], ref)
        r += m


# ------------------------------------------------------------- the ends of the cap --
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale,cap", [(0.1, 1e30), (-0.3, 1e30), (0.1, 1e-30), (0.0, 1e-30)])
def test_caps_at_both_ends_of_their_range(dtype, scale, cap):
    # the largest cap leaves the scores as they are, the smallest makes them 0
    P = Paged([300], 16, 2, 128, dtype)
    q = torch.randn(40, 8, 128, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    qs = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    ref = attend(q.double().cpu(), P.K[0], P.V[0], range(260, 300), scale if cap > 1 else 0.0, dtype=dtype)
    out, lse = E.paged_attn_prefill(q, qs, P.k, P.v, P.table, P.seq_len, scale, softcap=cap)
    check_rows("rows", out, lse, ref)
    out, lse = E.paged_attn_decode(q[-1:], P.k, P.v, P.table, P.seq_len, scale, softcap=cap)
    check_rows("token", out, lse, tuple(x[-1:] for x in ref))


# ----------------------------------------------------- numbers that no struct takes --
@pytest.mark.parametrize("kw", [dict(window=1 << 31), dict(window=1 << 40), dict(scale=1e39), dict(softcap=1e300)])
def test_numbers_past_the_structs_types_are_refused_like_others(kw):
    P = Paged([20, 9], 8, 2, 64, BF)
    q = torch.zeros(2, 4, 64, dtype=BF, device=DEV)
    kw = dict(dict(scale=0.1), **kw)
    qs = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    for call in (lambda: E.paged_attn_decode(q, P.k, P.v, P.table, P.seq_len, **kw),
                 lambda: E.paged_attn_prefill(q, qs, P.k, P.v, P.table, P.seq_len, **kw)):
        with pytest.raises(E.EchoError) as e:
            call()
        assert e.value.code == E.ERR_INVALID_ARG


# ------------------------------------------------ captured, with buffers of the call's own --
@pytest.mark.parametrize("given", ["none", "same", "forked"])
def test_captured_calls_with_default_buffers(given):
    """Append, rows and token captured with buffers of their own, on the capturing stream, named or
    not, or on one forked from it; replayed with other queries between other allocations."""
    Hq, Hkv, d, T = 16, 2, 128, 16
    P = Paged([5000, 300], T, Hkv, d, BF, seed=3)
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, h, d, generator=g).to(BF).to(DEV) for h in (Hq, Hkv, Hkv))
    qq = torch.randn(40, Hq, d, generator=g).to(BF).to(DEV)
    qs = torch.tensor([0, 30, 40], dtype=torch.int32, device=DEV)
    main, other = torch.cuda.Stream(), torch.cuda.Stream()
    stream = {"none": None, "same": main, "forked": other}[given]

    def calls(s):
        r = E.paged_append(k, v, P.k, P.v, P.table, P.seq_len, q=q, stream=s)
        a = E.paged_attn_prefill(qq, qs, P.k, P.v, P.table, P.seq_len, 0.1, stream=s)
        return (*a, *E.paged_attn_decode(r, P.k, P.v, P.table, P.seq_len, 0.1, stream=s))

    calls(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        if given == "forked":
            other.wait_stream(main)
        got = calls(stream)
        if given == "forked":
            main.wait_stream(other)
    for i in range(4):
        for x in (q, k, v, qq):
            x.normal_()
        want = [x.clone() for x in calls(None)]
        for x in got:
            x.fill_(7)
        graph.replay()
        junk = [torch.full((1 << 20,), 9.0, device=DEV) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        del junk
