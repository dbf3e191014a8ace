"""Refusals of the paged-cache calls that the library makes before any launch (no GPU)."""

import ctypes

import pytest

import sparse_attention_kv_dsa_gb300.echo as E

P = 1 << 20          # an aligned address that is never read


def cache(**kw):
    f = dict(k=P, v=P, page_stride=8 * 2 * 64, row_stride=2 * 64, head_stride=64, n_pages=4, page_tokens=8,
             n_kv_heads=2, head_dim=64, dtype=E.BF16, max_pages=3, page_table=P, status=None)
    f.update(kw)
    return E.PagedKVT(*f.values())


def scores(**kw):
    f = dict(scale=0.1, softcap=0.0, slopes=None, window=0, first_tok=None, prefix_len=None)
    f.update(kw)
    return E.AttnScoresT(*f.values())


def decode(c, s, q=P, q_stride=4 * 64, seq_len=P, B=2, Hq=4, out=P, lse=P, ws=P, nbytes=1 << 30):
    return E.lib().echo_paged_attn_decode(c and ctypes.byref(c), q, q_stride, seq_len, B, Hq, s and ctypes.byref(s), out,
                                          lse, ws, nbytes, None)


def prefill(c, s, q=P, q_stride=4 * 64, q_start=P, seq_len=P, N=5, B=2, Hq=4, out=P, lse=P, ws=P, nbytes=1 << 40):
    return E.lib().echo_paged_attn_prefill(c and ctypes.byref(c), q, q_stride, q_start, seq_len, N, B, Hq,
                                           s and ctypes.byref(s), out, lse, ws, nbytes, None)


def append(c, q=P, qs=256, k=P, ks=128, v=P, vs=128, q_out=P, q_start=P, seq_len=P, N=5, B=2, Hq=4, cs=P, max_pos=9,
           rot=64, inter=0):
    return E.lib().echo_paged_append(c and ctypes.byref(c), q, qs, k, ks, v, vs, q_out, q_start, seq_len, N, B, Hq, cs,
                                     max_pos, rot, inter, None)


INV, UNS = E.ERR_INVALID_ARG, E.ERR_UNSUPPORTED
BAD_CACHES = [(dict(k=None), INV), (dict(v=None), INV), (dict(page_table=None), INV), (dict(n_pages=0), INV),
              (dict(page_tokens=0), INV), (dict(n_kv_heads=0), INV), (dict(max_pages=-1), INV), (dict(k=P + 8), INV),
              (dict(v=P + 2), INV), (dict(row_stride=132), INV), (dict(head_stride=65), INV), (dict(page_stride=1), INV),
              (dict(head_dim=96), UNS), (dict(head_dim=256), UNS), (dict(dtype=E.E4M3), UNS), (dict(dtype=7), UNS),
              (dict(max_pages=1 << 30), UNS)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(kw, code):
    c = cache(**kw)
    assert decode(c, scores()) == code and prefill(c, scores()) == code and append(c) == code


@pytest.mark.parametrize("kw", [dict(scale=float("nan")), dict(scale=float("inf")), dict(softcap=-2.0),
                                dict(softcap=float("nan")), dict(window=-3)])
def test_bad_scores(kw):
    assert decode(cache(), scores(**kw)) == INV and prefill(cache(), scores(**kw)) == INV


def test_null_and_sizes():
    assert decode(None, scores()) == INV and decode(cache(), None) == INV
    for kw in (dict(q=None), dict(seq_len=None), dict(out=None), dict(lse=None), dict(ws=None), dict(B=0), dict(Hq=0),
               dict(q=P + 4), dict(q_stride=257), dict(out=P + 8), dict(nbytes=100), dict(ws=P + 4)):
        assert decode(cache(), scores(), **kw) == INV, kw
    for kw in (dict(Hq=3), dict(Hq=2 * 129)):
        assert decode(cache(), scores(), **kw) == UNS and prefill(cache(), scores(), **kw) == UNS, kw
    for kw in (dict(q=None), dict(q_start=None), dict(seq_len=None), dict(out=None), dict(lse=None), dict(N=0),
               dict(B=-1), dict(q=P + 4), dict(q_stride=257), dict(out=P + 8)):
        assert prefill(cache(), scores(), **kw) == INV, kw
    for kw in (dict(k=None), dict(v=None), dict(seq_len=None), dict(N=0), dict(B=0), dict(q=None), dict(q_out=None),
               dict(Hq=0), dict(q_start=None), dict(cs=None), dict(max_pos=0), dict(rot=-16), dict(k=P + 8), dict(ks=129),
               dict(vs=4), dict(qs=3), dict(q_out=P + 2)):
        assert append(cache(), **kw) == INV, kw
    for rot in (8, 24, 80, 128):
        assert append(cache(), rot=rot) == UNS


def test_work_that_32_bits_cannot_count():
    # 2^31 - 2^16 tokens of a sequence are the most that a table may hold; then 33.5M 64-token tiles
    big = dict(max_pages=32767, page_tokens=65536)
    assert decode(cache(max_pages=32768, page_tokens=65536), scores()) == UNS
    assert decode(cache(**big), scores(), B=1000) == UNS
    assert prefill(cache(**big), scores(), N=70000) == UNS
    assert prefill(cache(), scores(), N=2049, B=2049) == UNS
    assert prefill(cache(), scores(), N=0x7fffffff, nbytes=1 << 40) == UNS


def test_struct_layouts_and_workspaces():
    out = (ctypes.c_size_t * 2)()
    E.lib().echo_paged_struct_sizes(out)
    assert list(out) == [ctypes.sizeof(E.PagedKVT), ctypes.sizeof(E.AttnScoresT)]
    assert list(out) == [E._PAGED.size, E._SCORES.size]
    # the packed forms that the binding passes are the structs, field by field
    assert E._PAGED.pack(*range(1, 14)) == bytes(E.PagedKVT(*range(1, 14)))
    a, b = E._SCORES.pack(0.5, 2.0, 3, 4, 5, 6), bytes(E.AttnScoresT(0.5, 2.0, 3, 4, 5, 6))
    assert [a[i:i + 4] for i in (0, 4, 8, 16, 24, 32)] == [b[i:i + 4] for i in (0, 4, 8, 16, 24, 32)]
    assert E.paged_decode_workspace_bytes(64, 8, 128) > 0
    assert E.paged_decode_workspace_bytes(7, 2, 128) == 0
    # one bound for every batch and length: it depends on the heads alone
    assert E.paged_decode_workspace_bytes(64, 4, 128) == E.paged_decode_workspace_bytes(64, 2, 128)
