"""Paged attention over caches whose right answers are whole numbers, so that a single token lost,
taken twice or read from a wrong row shows, however long the sequence.

Keys are rows of random bits, and a query head is 0 or picks one of them; with a scale of ln 2 a
token weighs 2^bit: 1 or 2 (1 for the heads that are 0).  A token's value row holds one +1 or -1, at
a column drawn for each token and KV head; the tokens of a column take turns in sign.  So

  out[r, h, j] = S / W,   S = sum of weight * sign over the seen tokens of column j,   W = sum of weights,

with whole S and W.  A lost token, a wrong key bit or a wrong value row changes S by 1 at least.

The bounds.  Relative to a row's maximum weights are 1/2, 1 or 2, each off by 2^-22 of itself at
most (two to a power) and exact once rounded to bf16.
  S: bf16 adds exact halves, so it is exact.  float32: some 500 weights to a column, their sums
     below 2^10, each sum off by 2^-24 of that: 500 * 2^-14 = 2^-5.
  W: no float32 sum has more than 4000 steps in turn: 2^-12 of W, the weights' own 2^-22 in it.
  The quotient: half a step of the type (bf16 2^-8).  With |S| <= 110
  bf16: |out W - S| <= 110 (2^-8 + 2^-12) < 1/2: out W rounded to a whole number is S;
  float32: |out W - S| <= 2^-5 + 110 * 2^-11 < 1/4.
Heads that are 0 have weights of exactly 1 (2^0) and a W that float32 counts exactly, so
lse = ln W is off by two units of log2 W and one of the product: 4 * 2^-23 |lse| at most, where a
token more or less is 1 / W."""

import math

import numpy as np
import pytest
import torch

import sparse_attention_kv_dsa_gb300.echo as E

from paged_ref import DEV, Paged, doc_starts

BF, F32 = torch.bfloat16, torch.float32
LN2 = math.log(2.0)


def test_the_scale_is_one_in_base_2():
    assert np.float32(LN2) * np.float32(1.4426950408889634) == np.float32(1)


def codes(L, Hkv, d, seed):
    """Keys [L, Hkv, d] of bits and values [L, Hkv, d] of one +-1 a row."""
    g = torch.Generator().manual_seed(seed)
    K = torch.randint(0, 2, (L, Hkv, d), generator=g).double()
    col = torch.randint(0, d, (L, Hkv), generator=g)
    V = torch.zeros(L, Hkv, d, dtype=torch.float64)
    V.scatter_(2, col[:, :, None], 1.0)
    V = V * (1 - 2 * ((V.cumsum(0) - 1) % 2))            # every other token of a column is -1
    return K, V


def queries(N, Hq, Hkv, d, seed):
    """Query heads: the first of a KV head's group is 0, the others pick a bit, another in each row."""
    g = torch.Generator().manual_seed(seed)
    q = torch.zeros(N, Hq, d, dtype=torch.float64)
    q.scatter_(2, torch.randint(0, d, (N, Hq, 1), generator=g), 1.0)
    q[:, ::Hq // Hkv] = 0
    return q


def whole(q, K, V, see):
    """S [n, Hq, d] and W [n, Hq] for the seen tokens see [n, L]."""
    G = q.shape[1] // K.shape[1]
    S = torch.zeros(q.shape, dtype=torch.float64)
    W = torch.zeros(q.shape[:2], dtype=torch.float64)
    for h in range(q.shape[1]):
        w = torch.exp2(q[:, h] @ K[:, h // G].T) * see
        S[:, h], W[:, h] = w @ V[:, h // G], w.sum(1)
    assert float(S.abs().max()) <= 110
    return S, W


def sight(pos, L, window=0, prefix=0, first=None):
    t, p = torch.arange(L), torch.as_tensor(pos).view(-1, 1)
    see = (t <= p) & (t > p - window if window else t >= 0)
    see = see | (t < prefix)
    return see if first is None else see & (t >= torch.as_tensor(first).view(-1, 1))


def off(out, lse, S, W, q):
    """What is wrong with out and lse, or None."""
    dtype, some = out.dtype, W > 0
    o, z = out.double().cpu(), lse.double().cpu()
    if not torch.equal(torch.isneginf(z), ~some) or bool(o[~some].any()) or not bool(torch.isfinite(o).all()):
        return "empty rows"
    got = o * W[..., None]
    got = got.round() if dtype is BF else got
    if bool(((got - S).abs() > 0.25).any()):
        return f"{int(((got - S).abs() > 0.25).sum())} columns"
    count = some & (q == 0).all(2)
    if bool(((z - W.log()).abs() > 4 * 2.0 ** -23 * z.abs() + 1e-30)[count].any()):
        return "counts"
    return None


# ----------------------------------------------------------- the bounds themselves --
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L,d", [(60013, 128), (20011, 64)])
def test_the_bounds_tell_single_tokens(dtype, L, d):
    K, V = codes(L, 1, d, 1)
    q = queries(2, 4, 1, d, 2)
    see = sight([L - 1, L - 300], L)
    S, W = whole(q, K, V, see)

    def told(K=K, V=V, see=see):
        s, w = whole(q, K, V, see)
        return off((s / w[..., None]).float().to(dtype), w.log().float(), S, W, q)

    assert told() is None
    g = torch.Generator().manual_seed(3)
    for t in [0, 15, 16, L // 2, L - 302, *torch.randint(0, L - 310, (20,), generator=g).tolist()]:
        one = see.clone()
        one[:, t] = False
        assert told(see=one), f"token {t} lost"
        twice = see.double()
        twice[:, t] = 2
        assert told(see=twice), f"token {t} twice"
        other = next(o for o in range(L) if not torch.equal(V[o], V[t]))
        v = V.clone()
        v[t] = V[other]
        assert told(V=v), f"value row {t} of another token"
        k = K.clone()
        k[t] = 1 - K[t]
        assert told(K=k), f"key row {t} of another token"
    for n in (16, 64, 128, 384):
        tile = see.clone()
        tile[:, 5 * n:6 * n] = False
        assert told(see=tile), f"a tile of {n}"


# ------------------------------------------------------------------------ the kernels --
class Coded(Paged):
    def __init__(self, lens, T, Hkv, d, dtype, seed):
        super().__init__(lens, T, Hkv, d, dtype, seed=seed, fill=False)
        self.codes = [codes(n, Hkv, d, seed + b) for b, n in enumerate(lens)]
        for b, n in enumerate(lens):
            if n:
                pg, row = self.at(b, torch.arange(n))
                self.k[pg, row], self.v[pg, row] = (x.to(dtype).to(DEV) for x in self.codes[b])


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


MASKS = [dict(), dict(window=3001, prefix=61), dict(first=True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", MASKS)
@pytest.mark.parametrize("lens,T,Hq,Hkv,d", [([60013], 16, 8, 2, 128), ([30011], 24, 8, 1, 64), ([20011, 1, 0, 4099], 64, 40, 2, 128),
                                             ([9001, 17, 12007], 5, 9, 3, 64), ([777] * 150, 16, 4, 1, 64)])
def test_decode_counts_every_token_once(dtype, kw, lens, T, Hq, Hkv, d):
    P = Coded(lens, T, Hkv, d, dtype, 5)
    window, prefix = kw.get("window", 0), kw.get("prefix", 0)
    first = [n // 3 + 7 for n in lens] if kw.get("first") else None
    q = queries(len(lens), Hq, Hkv, d, 6)
    out, lse = E.paged_attn_decode(q.to(dtype).to(DEV), P.k, P.v, P.table, P.seq_len, LN2, window=window,
                                   first_tok=i32(first), prefix_len=i32([prefix] * len(lens)), status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    for b, n in enumerate(lens):
        see = sight([n - 1], n, window, prefix, None if first is None else [first[b]])
        S, W = whole(q[b:b + 1], *P.codes[b], see)
        assert off(out[b:b + 1], lse[b:b + 1], S, W, q[b:b + 1]) is None, f"sequence {b} of {n}"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", MASKS)
@pytest.mark.parametrize("lens,new,T,Hq,Hkv,d", [
    ([20011, 7003], [4, 3], 16, 8, 2, 128),                            # drafted tokens
    ([20011, 7003], [4, 3], 8, 16, 1, 64),
    ([12007], [300], 64, 8, 2, 128), ([9001], [200], 24, 6, 2, 64),    # chunks
    ([2311, 40, 700], [2311, 40, 700], 16, 4, 1, 128),                 # prompts
    ([1501], [1501], 5, 2, 1, 64)])
def test_prefill_counts_every_token_once(dtype, kw, lens, new, T, Hq, Hkv, d):
    P = Coded(lens, T, Hkv, d, dtype, 7)
    window, prefix, N = kw.get("window", 0), kw.get("prefix", 0), sum(new)
    first = None
    if kw.get("first"):
        first = [int(doc_starts(n, 500, b)[n - m + i]) for b, (n, m) in enumerate(zip(lens, new)) for i in range(m)]
    q = queries(N, Hq, Hkv, d, 8)
    out, lse = E.paged_attn_prefill(q.to(dtype).to(DEV), i32([0, *np.cumsum(new).tolist()]), P.k, P.v, P.table, P.seq_len,
                                    LN2, window=window, first_tok=i32(first), prefix_len=i32([prefix] * len(lens)),
                                    status=P.status)
    torch.cuda.synchronize()
    assert P.status.item() == E.OK
    r = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        s = slice(r, r + m)
        see = sight(range(n - m, n), n, window, prefix, None if first is None else first[s])
        S, W = whole(q[s], *P.codes[b], see)
        assert off(out[s], lse[s], S, W, q[s]) is None, f"sequence {b}: {m} of {n}"
        r += m
