"""Measured cases of the paged-cache operators: appending rotated keys and values to a
paged cache, attention of one new token per sequence over it, and attention of many new
tokens (prompts, chunks of prompts, a few drafted tokens) over it, with the tanh cap, the
distance bias and the window, document and prefix masks.

A case is one call.  `run` computes the plain form (elementary torch operations in 32
bits, rounded once) or, where `own` is true, calls the library.
"""

import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------- cases --
# op: "append", "decode" or "prefill"; B sequences of lo..hi cached tokens (the new ones
# among them), new_lo..new_hi of them new; Hq query heads, Hkv key/value heads of d values;
# page: tokens a page; heads_first: pages laid out [Hkv, page, d] instead of [page, Hkv, d];
# rot: rotated values of a head (interleaved or half-split pairs); cap, window, alibi, docs
# (mean tokens a document, 0 = no document mask), prefix (0 = none): the modifiers of scores.
def _case(name=None, *, op, B, lo, hi, Hq, Hkv, d, page, dtype="bf16", new_lo=1, new_hi=1, lens=1, heads_first=False,
          rot=0, interleaved=False, cap=0.0, window=0, alibi=False, docs=0, prefix=0):
    c = dict(op=op, B=B, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype, new_lo=new_lo, new_hi=new_hi,
             lens=lens, heads_first=heads_first, rot=rot, interleaved=interleaved, cap=cap, window=window, alibi=alibi,
             docs=docs, prefix=prefix)
    return c if name is None else dict(name=name, **c)


def listed():
    return [
        # one new token of each of eight requests at 20K tokens: launch latency decides
        _case("append-token-b8", op="append", B=8, lo=19000, hi=20480, Hq=64, Hkv=8, d=128, page=16, rot=128),
        # a batch of ragged prompts entering the cache, pages laid out heads first
        _case("append-prompt-8k", op="append", B=5, lo=900, hi=2600, new_lo=900, new_hi=2600, Hq=64, Hkv=8, d=128,
              page=64, rot=128, heads_first=True),
        # float32 chunks with half of each head rotated, neighbouring pairs, an odd page size
        _case("append-chunk-f32", op="append", B=3, lo=2000, hi=4500, new_lo=300, new_hi=700, Hq=12, Hkv=4, d=64,
              page=24, rot=32, interleaved=True, dtype="f32"),
        # one request alone: the latency of a single user's token
        _case("decode-b1-ctx8k", op="decode", B=1, lo=8100, hi=8192, Hq=64, Hkv=8, d=128, page=16),
        # the saturated batch of the GQA workload: 16 requests of 32K to 48K tokens
        _case("decode-b16-ctx32k-48k", op="decode", B=16, lo=32768, hi=49152, Hq=64, Hkv=8, d=128, page=16),
        # many short and middling requests, capped scores, a window with kept first tokens
        _case("decode-b96-capped-window", op="decode", B=96, lo=70, hi=9000, Hq=40, Hkv=8, d=64, page=64, cap=50.0,
              window=4096, prefix=4),
        # float32 with a distance bias
        _case("decode-b4-f32-alibi", op="decode", B=4, lo=2500, hi=4096, Hq=32, Hkv=8, d=128, page=32, dtype="f32",
              alibi=True),
        # one whole prompt: the tensor rate decides
        _case("prefill-1x8192", op="prefill", B=1, lo=8192, hi=8192, new_lo=8192, new_hi=8192, Hq=64, Hkv=8, d=128,
              page=16),
        # a chunk of a long prompt against what is cached, capped scores
        _case("prefill-chunk512-ctx32k-capped", op="prefill", B=1, lo=32768, hi=32768, new_lo=512, new_hi=512, Hq=32,
              Hkv=8, d=128, page=64, cap=30.0),
        # ragged packed prompts made of documents that do not see one another, distance bias
        _case("prefill-ragged-docs-alibi", op="prefill", B=8, lo=130, hi=1500, new_lo=130, new_hi=1500, Hq=16, Hkv=2,
              d=64, page=16, alibi=True, docs=300),
        # four drafted tokens of each request checked in one pass
        _case("prefill-draft4-b16-ctx20k", op="prefill", B=16, lo=17000, hi=20480, new_lo=4, new_hi=4, Hq=64, Hkv=8,
              d=128, page=16),
        # float32, prompts whose first tokens see one another both ways
        _case("prefill-f32-prefix", op="prefill", B=2, lo=600, hi=1100, new_lo=600, new_hi=1100, Hq=8, Hkv=4, d=64,
              page=16, dtype="f32", prefix=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    d = rng.choice([64, 128])
    f32 = rng.random() < 0.2
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16])
    G = G if Hkv * G <= 64 else 64 // Hkv
    page = rng.choice([8, 16, 20, 32, 64, 128])
    kw = dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, dtype="f32" if f32 else "bf16", lens=rng.randrange(1, 1 << 30),
              heads_first=rng.random() < 0.3)
    if op == "append":
        rot = rng.choice([d, d, d // 2, 0])
        if rng.random() < 0.5:
            hi = _log(rng, 2, 40000)
            kw.update(B=_log(rng, 1, 128), lo=max(1, hi // 2), hi=hi)
        else:
            hi = _log(rng, 16, 6000)
            kw.update(B=rng.randrange(1, 4), lo=hi, hi=2 * hi, new_lo=max(1, hi // 3), new_hi=hi)
        return _case(rot=rot, interleaved=rng.random() < 0.4, **kw)
    kw.update(cap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.25)
    if op == "decode":
        B = _log(rng, 1, 96)
        hi = _log(rng, 2, min(48000, max(64, 600000 // B)) // (4 if f32 else 1))
        kw.update(B=B, lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, window=rng.choice([0, 0, 0, _log(rng, 64, 8192)]))
        kw.update(prefix=rng.choice([0, 4, 61]) if kw["window"] else 0)
        return _case(**kw)
    B = _log(rng, 1, 8)
    new = _log(rng, 2, (400 if f32 else 4000) // B + 2)
    ctx = new + (_log(rng, 1, min(2000 if f32 else 30000, 24000000 // (B * new))) if rng.random() < 0.5 else 0)
    mask = rng.choice(["none", "none", "window", "docs", "prefix"])
    kw.update(window=_log(rng, 16, 4096) if mask == "window" else 0, docs=_log(rng, 30, 1000) if mask == "docs" else 0,
              prefix=_log(rng, 2, max(3, ctx)) if mask == "prefix" else 0)
    return _case(B=B, lo=ctx, hi=ctx + new // 2, new_lo=max(1, new // 2), new_hi=new, **kw)


# ------------------------------------------------------------------ a case's plan --
def _plan(c):
    """Lengths, new tokens, document starts and prefixes of a case (from the case alone)."""
    r = np.random.RandomState(c["lens"] % (1 << 31))
    B = c["B"]
    new = r.randint(c["new_lo"], c["new_hi"] + 1, B)
    lens = r.randint(c["lo"], c["hi"] + 1, B)
    whole = c["lo"] == c["new_lo"] and c["hi"] == c["new_hi"] and c["op"] != "decode"
    lens = new.copy() if whole else np.maximum(lens, new)
    q_start = np.concatenate([[0], np.cumsum(new)])
    seq = np.repeat(np.arange(B), new)
    pos = np.arange(q_start[-1]) - q_start[seq] + (lens - new)[seq]
    first = np.zeros_like(pos)
    if c["docs"]:
        for b in range(B):
            cuts = np.sort(r.randint(0, lens[b], max(1, int(lens[b] // c["docs"]))))
            cuts = np.concatenate([[0], cuts])
            at = pos[seq == b]
            first[seq == b] = cuts[np.searchsorted(cuts, at, side="right") - 1]
    prefix = np.minimum(np.full(B, c["prefix"]), lens)
    return dict(lens=lens, new=new, q_start=q_start, seq=seq, pos=pos, first=first, prefix=prefix)


def _sizes(c, p):
    pages = -(-p["lens"] // c["page"])
    max_pages = int(pages.max()) + 1
    n_pages = int(pages.sum()) + 3
    return pages, max_pages, n_pages


def work(case):
    c, p = case, _plan(case)
    es = 2 if c["dtype"] == "bf16" else 4
    N, B = int(p["q_start"][-1]), c["B"]
    if c["op"] == "append":
        rows = 2 * N * (c["Hq"] + 2 * c["Hkv"]) * c["d"] * es
        return {"bytes": rows + N * (c["rot"] * 4 + 4) + 8 * B, "flops": 3 * N * (c["Hq"] + c["Hkv"]) * c["rot"]}
    L, pre, first, pos = p["lens"][p["seq"]], p["prefix"][p["seq"]], p["first"], p["pos"]
    start = np.maximum(first, pos - c["window"] + 1) if c["window"] else first
    start = np.maximum(start, 0)
    a = np.maximum(np.minimum(pre, L) - first, 0)                       # seen through the prefix
    seen = np.maximum(pos + 1 - start, 0) + a
    seen -= np.maximum(np.minimum(pos + 1, np.minimum(pre, L)) - start, 0)   # counted twice
    # cached tokens that some row sees
    kv = 0
    for b in range(B):
        m = p["seq"] == b
        lo, hi = int(start[m].min()), int(pos[m].max()) + 1
        f, e = int(first[m].min()), int(min(p["prefix"][b], p["lens"][b]))
        kv += hi - lo + max(0, e - f) - max(0, min(hi, e) - max(lo, f))
    bytes_ = kv * 2 * c["Hkv"] * c["d"] * es + 2 * N * c["Hq"] * c["d"] * es + 4 * N * c["Hq"]
    bytes_ += 4 * kv // c["page"] + 12 * B
    return {"bytes": int(bytes_), "flops": int(seen.sum()) * 4 * c["d"] * c["Hq"]}


# ------------------------------------------------------------------------- inputs --
def prepare(case, seed):
    c, p = case, _plan(case)
    pages, max_pages, n_pages = _sizes(c, p)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    N, B, T, Hq, Hkv, d = int(p["q_start"][-1]), c["B"], c["page"], c["Hq"], c["Hkv"], c["d"]

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device=dev).normal_(generator=g)

    def pool():
        x = normal(n_pages, Hkv, T, d) if c["heads_first"] else normal(n_pages, T, Hkv, d)
        return x.transpose(1, 2) if c["heads_first"] else x

    s = dict(op=c["op"], k_pages=pool(), v_pages=pool())
    # the pages of a pool in use lie in any order
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).cpu().numpy()
    table = np.full((B, max_pages), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += int(pages[b])

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)

    s.update(page_table=i32(table), seq_len=i32(p["lens"]), q_start=i32(p["q_start"]) if c["op"] != "decode" else None,
             scale=d ** -0.5, cap=c["cap"], window=c["window"])
    if c["op"] == "append":
        # the projections' fused output: a token's query, key and value heads side by side
        qkv = normal(N, Hq + 2 * Hkv, d)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], interleaved=c["interleaved"], cos_sin=None)
        s["q_start"] = None if int(p["new"].max()) == 1 else s["q_start"]
        s["q_out"] = torch.empty(N, Hq, d, dtype=dt, device=dev)
        if c["rot"]:
            half = c["rot"] // 2
            f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
            a = torch.arange(int(p["lens"].max()) + 1, dtype=torch.float64, device=dev)[:, None] * f
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        return s
    # some heads attend sharply, most of them broadly
    sharp = torch.where(torch.arange(Hq, device=dev) % 4 == 3, 3.0, 1.0).to(dt)
    s["q"] = normal(N, Hq, d) * sharp[:, None]
    s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq)).float() if c["alibi"] else None
    s["first_tok"] = i32(p["first"]) if c["docs"] else None
    s["prefix_len"] = i32(p["prefix"]) if c["prefix"] else None
    return s


# ---------------------------------------------------------------- the plain forms --
def _rows(s, N, B, dev):
    """Sequence and position of each row, and each row's place in its sequence."""
    start = s["q_start"] if s["q_start"] is not None else torch.arange(B + 1, dtype=torch.int32, device=dev)
    start = start.long()
    i = torch.arange(N, device=dev)
    seq = torch.searchsorted(start, i, right=True) - 1
    local = i - start[seq]
    pos = s["seq_len"].long()[seq] - (start[1:] - start[:-1])[seq] + local
    return start, seq, local, pos


def _rotated(x, cs, interleaved):
    x = x.float()
    r = cs.shape[1]
    cos, sin = cs[:, None, :r // 2], cs[:, None, r // 2:]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    ab = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([ab, x[..., r:]], -1)


def _append(s):
    q, k, v, kp, vp = s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"]
    N, B, T = q.shape[0], s["seq_len"].shape[0], kp.shape[1]
    _, seq, _, pos = _rows(s, N, B, q.device)
    if s["cos_sin"] is not None:
        cs = s["cos_sin"][pos]
        q, k = _rotated(q, cs, s["interleaved"]).to(q.dtype), _rotated(k, cs, s["interleaved"]).to(k.dtype)
    page = s["page_table"][seq, pos // T].long()
    kp[page, pos % T] = k
    vp[page, pos % T] = v
    s["q_out"].copy_(q)
    return s["q_out"], kp, vp


def _attend(s):
    q, kp, vp, table = s["q"], s["k_pages"], s["v_pages"], s["page_table"]
    N, Hq, d = q.shape
    B, T, Hkv = table.shape[0], kp.shape[1], kp.shape[2]
    G, L = Hq // Hkv, table.shape[1] * T
    start, seq, local, pos = _rows(s, N, B, q.device)
    n = int(N) if B == 1 else int((start[1:] - start[:-1]).max())       # rows of the padded batch
    rows = (start[:-1, None] + torch.arange(n, device=q.device)).clamp(max=N - 1)
    pages = table.clamp(min=0).long()
    K = kp[pages].reshape(B, L, Hkv, d).transpose(1, 2).float()
    V = vp[pages].reshape(B, L, Hkv, d).transpose(1, 2).float()
    Q = q[rows].float().reshape(B, n, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, n * G, d)
    x = (Q @ K.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, n, G, L)
    if s["cap"]:
        x = x.div_(s["cap"]).tanh_().mul_(s["cap"])
    t = torch.arange(L, device=q.device)
    at = pos[rows][:, :, None]                                          # [B, n, 1]
    if s["slopes"] is not None:
        far = (at - t).abs().float()[:, None, :, None, :]
        x = x.sub_(far * s["slopes"].view(1, Hkv, 1, G, 1))
    seen = t <= at
    if s["window"]:
        seen = seen & (t > at - s["window"])
    if s["prefix_len"] is not None:
        seen = seen | (t < s["prefix_len"][:, None, None])
    seen = seen & (t < s["seq_len"][:, None, None])
    if s["first_tok"] is not None:
        seen = seen & (t >= s["first_tok"][rows][:, :, None])
    x = x.masked_fill_(~seen[:, None, :, None, :], -math.inf).view(B, Hkv, n * G, L)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    V = V * (t < s["seq_len"][:, None])[:, None, :, None]
    o = (x @ V) / total.clamp(min=1e-38)
    lse = (m + total.log()).view(B, Hkv, n, G).transpose(1, 2).reshape(B, n, Hq)
    o = o.view(B, Hkv, n, G, d).transpose(1, 2).reshape(B, n, Hq, d)
    return o[seq, local].to(q.dtype), lse[seq, local].contiguous()


# ------------------------------------------------------------ the library's calls --
def _own(s):
    from sparse_attention_kv_dsa_gb300 import echo as E
    if s["op"] == "append":
        E.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_len"], q=s["q"],
                       q_out=s["q_out"], cos_sin=s["cos_sin"], interleaved=s["interleaved"], q_start=s["q_start"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    if s["op"] == "decode":
        return E.paged_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_len"], s["scale"],
                                   softcap=s["cap"], window=s["window"], slopes=s["slopes"],
                                   first_tok=s["first_tok"], prefix_len=s["prefix_len"])
    return E.paged_attn_prefill(s["q"], s["q_start"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_len"],
                                s["scale"], softcap=s["cap"], window=s["window"], slopes=s["slopes"],
                                first_tok=s["first_tok"], prefix_len=s["prefix_len"])


def run(state):
    if own:
        return _own(state)
    return _append(state) if state["op"] == "append" else _attend(state)


# -------------------------------------------------------------- 64-bit definition --
def exact(case, seed):
    c, p, s = case, _plan(case), prepare(case, seed)
    kp, vp, T = s["k_pages"], s["v_pages"], c["page"]
    table = s["page_table"].cpu().numpy()
    if c["op"] == "append":
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        pos = torch.from_numpy(p["pos"]).to(q.device)
        if c["rot"]:
            half = c["rot"] // 2
            # the angles are an input: the table's values, complex numbers of modulus 1
            cs = s["cos_sin"].double()[pos]
            z = torch.complex(cs[:, :half], cs[:, half:])[:, None]
            for x in (q, k):
                y = x[..., :c["rot"]]
                if c["interleaved"]:
                    w = torch.view_as_complex(y.reshape(*y.shape[:-1], half, 2).contiguous()) * z
                    x[..., :c["rot"]] = torch.view_as_real(w).reshape(y.shape)
                else:
                    w = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * z
                    x[..., :half], x[..., half:c["rot"]] = w.real, w.imag
        K, V = kp.double(), vp.double()
        page = torch.from_numpy(table[p["seq"], p["pos"] // T].astype(np.int64)).to(q.device)
        row = torch.from_numpy(p["pos"] % T).to(q.device)
        K[page, row], V[page, row] = k, v
        return q, K, V
    q, Hkv, d = s["q"].double(), c["Hkv"], c["d"]
    N, Hq = q.shape[0], q.shape[1]
    G = Hq // Hkv
    out = torch.zeros(N, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(c["B"]):
        L, r0, r1 = int(p["lens"][b]), int(p["q_start"][b]), int(p["q_start"][b + 1])
        ids = torch.from_numpy(table[b, :-(-L // T)].astype(np.int64)).to(q.device)
        t = torch.arange(L, device=q.device)[None]
        at = torch.from_numpy(p["pos"][r0:r1]).to(q.device)[:, None]
        see = t <= at
        if c["window"]:
            see = see & (at - t < c["window"])
        if c["prefix"]:
            see = see | (t < int(p["prefix"][b]))
        if c["docs"]:
            see = see & (t >= torch.from_numpy(p["first"][r0:r1]).to(q.device)[:, None])
        hide = torch.where(see, 0.0, -math.inf).double()
        for h in range(Hkv):
            K = kp[ids, :, h].reshape(-1, d)[:L].double()
            V = vp[ids, :, h].reshape(-1, d)[:L].double()
            for i in range(h * G, h * G + G):
                x = torch.einsum("nd,ld->nl", q[r0:r1, i], K) * s["scale"]
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["alibi"]:
                    x = x - float(s["slopes"][i]) * (at - t).abs()
                x = x + hide
                z = torch.logsumexp(x, 1)
                lse[r0:r1, i] = z
                out[r0:r1, i] = torch.exp(x - z[:, None]) @ V
    return out, lse
