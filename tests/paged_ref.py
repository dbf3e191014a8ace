"""Plain 64-bit forms of the paged-cache calls and the error bounds of their kernels."""

from __future__ import annotations

import math

import numpy as np
import torch

DEV = "cuda"


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


class Paged:
    """A pool with every row NaN except what `fill` or the library writes, and page tables of
    B sequences whose pages lie in random order."""

    def __init__(self, lens, T, Hkv, d, dtype, *, seed=0, heads_first=False, room=None, extra_pages=2, fill=True):
        g = torch.Generator().manual_seed(seed)
        self.T, self.Hkv, self.d, self.dtype = T, Hkv, d, dtype
        self.lens = list(lens)
        room = room or self.lens
        npg = [-(-r // T) for r in room]
        self.n_pages = sum(npg) + extra_pages
        shape = (self.n_pages, Hkv, T, d) if heads_first else (self.n_pages, T, Hkv, d)
        self.k, self.v = (torch.full(shape, math.nan, dtype=dtype, device=DEV) for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        order = torch.randperm(self.n_pages, generator=g).tolist()
        table = torch.full((len(self.lens), max(npg + [1]) + 1), -1, dtype=torch.int32)
        for b, n in enumerate(npg):
            table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
        self.table = table.to(DEV)
        self.seq_len = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.K, self.V = [], []                      # dense copies, float64
        for b, n in enumerate(self.lens):
            k, v = (torch.randn(n, Hkv, d, generator=g).to(dtype) for _ in range(2))
            self.K.append(k.double())
            self.V.append(v.double())
            if fill and n:
                pg, row = self.at(b, torch.arange(n))
                self.k[pg, row] = k.to(DEV)
                self.v[pg, row] = v.to(DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def at(self, b, t):
        t = t.to(DEV)
        return self.table[b, t // self.T].long(), t % self.T


def rotate(x, cs, interleaved):
    """Float64 rotation of x [N, H, d] by cs [N, rot] (cosines, then sines)."""
    x = x.double().clone()
    r = cs.shape[1]
    c, s = cs[:, None, :r // 2].double(), cs[:, None, r // 2:].double()
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def cos_sin(max_pos, rot):
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def attend(q, K, V, pos, scale, *, dtype, cap=0.0, window=0, slopes=None, first=None, prefix=0):
    """One sequence: q [n, Hq, d] float64 at positions pos [n], K, V [L, Hkv, d] float64 ->
    (out, lse, bound of out, bound of lse), [n, Hq, d] and [n, Hq].

    The bounds.  A score x = scale q.k in float32: d products and sums, each off by at most
    2^-24 of sum |q_i k_i|; the scale, the cap (its tanh within 2^-22 of the cap, see the
    kernel), the bias and the change to base 2 are some ten further roundings of magnitudes
    up to |x| + cap + |bias|: eps_x.  Two to a power: 2^-22.  A sum over n tokens: n 2^-24.
    So weights are off by e = 2 eps_x + 2^-21 + 2 n 2^-24 relative to their sum, and the
    result by e * sum p|v|; in bf16 every weight is rounded too (half a step of sum p|v|), and
    the result is rounded to its type."""
    n, Hq, d = q.shape
    L, Hkv = K.shape[0], K.shape[1]
    G = Hq // Hkv
    t = torch.arange(L)
    p = torch.as_tensor(pos).view(-1, 1)
    see = t <= p
    if window:
        see = see & (t > p - window)
    see = see | (t < prefix)
    if first is not None:
        see = see & (t >= torch.as_tensor(first).view(-1, 1))
    out, lse = torch.zeros(n, Hq, d, dtype=torch.float64), torch.full((n, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    some = see.any(1)
    hs = half_step(dtype)
    for h in range(Hq):
        k, v = K[:, h // G], V[:, h // G]
        x = (q[:, h] @ k.T) * scale
        mag = (q[:, h].abs() @ k.abs().T) * abs(scale) * d
        if cap:
            x = cap * torch.tanh(x / cap)
            mag = mag + 40 * cap
        if slopes is not None:
            far = float(slopes[h]) * (p - t).abs()
            x = x - far
            mag = mag + 10 * far
        x = x.masked_fill(~see, -math.inf)
        mag = (mag + 10 * x.abs().masked_fill(~see, 0)).masked_fill(~see, 0)
        z = torch.logsumexp(x, 1)
        w = torch.exp(x - torch.where(some, z, torch.zeros_like(z))[:, None])
        eps_x = mag.amax(1) * 2.0 ** -24 if L else torch.zeros(n)
        e = 2 * eps_x + 2.0 ** -21 + 2 * see.sum(1) * 2.0 ** -24
        out[:, h], lse[:, h] = w @ v, z
        a = w @ v.abs()
        tol[:, h] = e[:, None] * a + (hs * a if dtype == torch.bfloat16 else 0) + 1.01 * hs * out[:, h].abs() + 1e-30
        ltol[:, h] = e + 2.0 ** -22 * z.abs().masked_fill(~some, 0)
    return out, lse, tol, ltol


def check_rows(name, out, lse, ref):
    """Rows of the library against attend()'s."""
    o, z, tol, ltol = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    empty = torch.isneginf(z)
    assert torch.equal(torch.isneginf(lse), empty), f"{name}: rows that see nothing"
    assert not out[empty].any(), f"{name}: empty rows are zero"
    assert bool(torch.isfinite(out).all()), f"{name}: finite"
    bad = ((out - o).abs() / tol).max().item() if out.numel() else 0.0
    assert bad <= 1, f"{name}: out is {bad:.3g} of its bound off"
    f = ~empty
    bad = ((lse[f] - z[f]).abs() / ltol[f]).max().item() if f.any() else 0.0
    assert bad <= 1, f"{name}: lse is {bad:.3g} of its bound off"


def doc_starts(n, every, seed=0):
    """First position of the document of each position: documents of 1 .. 2 every tokens."""
    r = np.random.RandomState(seed)
    cuts, at = [0], 0
    while at < n:
        at += int(r.randint(1, 2 * every + 1))
        cuts.append(at)
    cuts = np.array(cuts)
    return cuts[np.searchsorted(cuts, np.arange(n), side="right") - 1]
