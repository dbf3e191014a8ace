"""Scales and caps whose scores float32 cannot form are refused before any launch (no GPU)."""

import ctypes

import pytest

import sparse_attention_kv_dsa_gb300.echo as E

P = 1 << 20          # an aligned address that is never read


def calls(**kw):
    c = E.PagedKVT(k=P, v=P, page_stride=8 * 2 * 64, row_stride=2 * 64, head_stride=64, n_pages=4, page_tokens=8,
                   n_kv_heads=2, head_dim=64, dtype=E.BF16, max_pages=3, page_table=P, status=None)
    s = E.AttnScoresT(**dict(dict(scale=0.1, softcap=0.0, window=0), **kw))
    L, c, s = E.lib(), ctypes.byref(c), ctypes.byref(s)
    return (L.echo_paged_attn_decode(c, P, 256, P, 2, 4, s, P, P, P, 1 << 30, None),
            L.echo_paged_attn_prefill(c, P, 256, P, P, 5, 2, 4, s, P, P, P, 1 << 40, None))


@pytest.mark.parametrize("kw", [dict(softcap=1e31), dict(softcap=1e38), dict(softcap=1e-31), dict(softcap=1e-39),
                                dict(scale=0.0, softcap=1e-40), dict(scale=1e30, softcap=1e-20),
                                dict(scale=-1e30, softcap=1e-20), dict(scale=3e38), dict(scale=-3e38)])
def test_scores_that_float32_cannot_form(kw):
    assert calls(**kw) == (E.ERR_INVALID_ARG, E.ERR_INVALID_ARG)
