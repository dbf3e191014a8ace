"""Measured cases of the paged cache in 8 bits and of head norms: appending keys and values
whose heads are normed and rotated in the same pass, to a cache in the activations' type or,
quantised row by row, to one of e4m3 codes; attention of one new token per sequence, and of
many, over the quantised cache.

A case is one call.  `run` computes the plain form (elementary torch operations in 32 bits,
rounded once) or, where `own` is true, calls the library.

The quantised cache: a row (the d values of one token's key or value head) holds e4m3 codes
and an exponent e in -64 .. 64, the smallest with max|x| <= 448 * 2^e; code = e4m3(x * 2^-e).
The exponents are held as float8_e8m0fnu, the number 2^e.
"""

import math

import numpy as np
import torch

own = False

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------------- cases --
# op: "append" (cache of dtype), "append_q8", "decode_q8" or "prefill_q8" (cache of e4m3, q of
# bf16); B sequences of lo..hi cached tokens (the new ones among them), new_lo..new_hi of them
# new; Hq query heads, Hkv key/value heads of d values; page: tokens a page; heads_first: pages
# and exponents laid out [Hkv, page] instead of [page, Hkv]; norm: query and key heads are
# normed; rot: rotated values of a head (interleaved or half-split pairs); cap, window, alibi,
# docs (mean tokens a document, 0 = no document mask), prefix (0 = none): modifiers of scores.
def _case(name=None, *, op, B, lo, hi, Hq, Hkv, d, page, dtype="bf16", new_lo=1, new_hi=1, lens=1, heads_first=False,
          norm=False, rot=0, interleaved=False, cap=0.0, window=0, alibi=False, docs=0, prefix=0):
    c = dict(op=op, B=B, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype, new_lo=new_lo, new_hi=new_hi,
             lens=lens, heads_first=heads_first, norm=norm, rot=rot, interleaved=interleaved, cap=cap, window=window,
             alibi=alibi, docs=docs, prefix=prefix)
    return c if name is None else dict(name=name, **c)


def listed():
    return [
        # one new token of each of sixteen requests, normed heads: launch latency decides
        _case("append-norm-token-b16", op="append", B=16, lo=19000, hi=20480, Hq=64, Hkv=8, d=128, page=16, norm=True,
              rot=128),
        # a batch of ragged prompts entering the cache, normed heads
        _case("append-norm-prompt-8k", op="append", B=5, lo=900, hi=2600, new_lo=900, new_hi=2600, Hq=64, Hkv=8, d=128,
              page=64, norm=True, rot=128),
        # one new token of each of eight requests into the quantised cache
        _case("append-q8-token-b8", op="append_q8", B=8, lo=19000, hi=20480, Hq=64, Hkv=8, d=128, page=16, rot=128),
        # ragged prompts, normed, rotated and quantised in one pass, pages laid out heads first
        _case("append-q8-norm-prompt-8k", op="append_q8", B=5, lo=900, hi=2600, new_lo=900, new_hi=2600, Hq=64, Hkv=8,
              d=128, page=64, norm=True, rot=128, heads_first=True),
        # chunks with half of each head rotated, neighbouring pairs, an odd page size
        _case("append-q8-chunk-d64", op="append_q8", B=3, lo=2000, hi=4500, new_lo=300, new_hi=700, Hq=12, Hkv=4, d=64,
              page=24, rot=32, interleaved=True),
        # one request alone: the latency of a single user's token
        _case("decode-q8-b1-ctx8k", op="decode_q8", B=1, lo=8100, hi=8192, Hq=64, Hkv=8, d=128, page=16),
        # the saturated batch of the GQA workload: 16 requests of 32K to 48K tokens
        _case("decode-q8-b16-ctx32k-48k", op="decode_q8", B=16, lo=32768, hi=49152, Hq=64, Hkv=8, d=128, page=16,
              heads_first=True),
        # many short and middling requests, capped scores, a window with kept first tokens
        _case("decode-q8-b96-capped-window", op="decode_q8", B=96, lo=70, hi=9000, Hq=40, Hkv=8, d=64, page=64,
              cap=50.0, window=4096, prefix=4),
        # one whole prompt: the tensor rate decides
        _case("prefill-q8-1x8192", op="prefill_q8", B=1, lo=8192, hi=8192, new_lo=8192, new_hi=8192, Hq=64, Hkv=8,
              d=128, page=16),
        # a chunk of a long prompt against what is cached, capped scores
        _case("prefill-q8-chunk512-ctx32k-capped", op="prefill_q8", B=1, lo=32768, hi=32768, new_lo=512, new_hi=512,
              Hq=32, Hkv=8, d=128, page=64, cap=30.0, heads_first=True),
        # ragged packed prompts made of documents that do not see one another, distance bias
        _case("prefill-q8-ragged-docs-alibi", op="prefill_q8", B=8, lo=130, hi=1500, new_lo=130, new_hi=1500, Hq=16,
              Hkv=2, d=64, page=16, alibi=True, docs=300),
        # four drafted tokens of each request checked in one pass
        _case("prefill-q8-draft4-b16-ctx20k", op="prefill_q8", B=16, lo=17000, hi=20480, new_lo=4, new_hi=4, Hq=64,
              Hkv=8, d=128, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append_q8", "decode_q8", "decode_q8", "prefill_q8", "prefill_q8"])
    d = rng.choice([64, 128])
    f32 = op == "append" and rng.random() < 0.3
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16])
    G = G if Hkv * G <= 64 else 64 // Hkv
    page = rng.choice([8, 16, 20, 32, 64, 128])
    kw = dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, dtype="f32" if f32 else "bf16", lens=rng.randrange(1, 1 << 30),
              heads_first=rng.random() < 0.4)
    if op.startswith("append"):
        rot = rng.choice([d, d, d // 2, 0])
        if rng.random() < 0.5:
            hi = _log(rng, 2, 40000)
            kw.update(B=_log(rng, 1, 128), lo=max(1, hi // 2), hi=hi)
        else:
            hi = _log(rng, 16, 6000)
            kw.update(B=rng.randrange(1, 4), lo=hi, hi=2 * hi, new_lo=max(1, hi // 3), new_hi=hi)
        return _case(rot=rot, interleaved=rng.random() < 0.4, norm=op == "append" or rng.random() < 0.5, **kw)
    kw.update(cap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.25)
    if op == "decode_q8":
        B = _log(rng, 1, 96)
        hi = _log(rng, 2, min(48000, max(64, 600000 // B)))
        kw.update(B=B, lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, window=rng.choice([0, 0, 0, _log(rng, 64, 8192)]))
        kw.update(prefix=rng.choice([0, 4, 61]) if kw["window"] else 0)
        return _case(**kw)
    B = _log(rng, 1, 8)
    new = _log(rng, 2, 4000 // B + 2)
    ctx = new + (_log(rng, 1, min(30000, 24000000 // (B * new))) if rng.random() < 0.5 else 0)
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
    whole = c["lo"] == c["new_lo"] and c["hi"] == c["new_hi"] and c["op"] != "decode_q8"
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
    N, B, d = int(p["q_start"][-1]), c["B"], c["d"]
    if c["op"].startswith("append"):
        read = N * (c["Hq"] + 2 * c["Hkv"]) * d * es + N * (c["rot"] * 4 + 4) + 8 * B + (2 * d * es if c["norm"] else 0)
        kept = N * 2 * c["Hkv"] * (d + 1 if c["op"] == "append_q8" else d * es)
        flops = 3 * N * (c["Hq"] + c["Hkv"]) * c["rot"] + (4 * N * (c["Hq"] + c["Hkv"]) * d if c["norm"] else 0)
        flops += 2 * N * 2 * c["Hkv"] * d if c["op"] == "append_q8" else 0
        return {"bytes": read + N * c["Hq"] * d * es + kept, "flops": flops}
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
    bytes_ = kv * 2 * c["Hkv"] * (d + 1) + 2 * N * c["Hq"] * d * es + 4 * N * c["Hq"]
    bytes_ += 4 * kv // c["page"] + 12 * B
    return {"bytes": int(bytes_), "flops": int(seen.sum()) * 4 * d * c["Hq"]}


# ------------------------------------------------------------- rows in 8 bits, plain --
def _exponent(x):
    """The exponent of rows x [..., d] (float32): max|x| <= 448 * 2^e, the smallest in -64 .. 64."""
    m, k = torch.frexp(x.abs().amax(-1))                                # max = m 2^k, 0.5 <= m < 1
    e = k - 9 + (m > 0.875).int()                                       # 448 = 0.875 * 2^9
    return torch.where(m == 0, -64, e).clamp(-64, 64)


def _codes(x, e):
    return torch.ldexp(x, -e[..., None]).clamp(-448, 448).to(F8)


def _e8(e):
    return (e + 127).to(torch.uint8).view(E8)


def _two_to(s):
    """The numbers 2^e that exponents stand for, float32."""
    return torch.exp2(s.view(torch.uint8).float() - 127)


# ------------------------------------------------------------------------- inputs --
def prepare(case, seed):
    c, p = case, _plan(case)
    pages, max_pages, n_pages = _sizes(c, p)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    N, B, T, Hq, Hkv, d = int(p["q_start"][-1]), c["B"], c["page"], c["Hq"], c["Hkv"], c["d"]
    q8 = c["op"] != "append"

    def normal(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)

    shape = (n_pages, Hkv, T, d) if c["heads_first"] else (n_pages, T, Hkv, d)

    def flip(x):
        return x.transpose(1, 2) if c["heads_first"] else x

    def pool():
        if not q8:
            return flip(normal(*shape)), None
        # rows of differing size with some large channels, in 8 bits
        codes, exps = torch.empty(shape, dtype=F8, device=dev), torch.empty(shape[:3], dtype=torch.uint8, device=dev).view(E8)
        big = 1 + 7 * (torch.rand(d, generator=g, device=dev) < 0.06).float()
        for i in range(0, n_pages, 4096):
            x = normal(*codes[i:i + 4096].shape, dtype=torch.float32) * big
            x = x * torch.exp2(normal(*x.shape[:3], 1, dtype=torch.float32) * 0.7)
            e = _exponent(x)
            codes[i:i + 4096], exps.view(torch.uint8)[i:i + 4096] = _codes(x, e), _e8(e).view(torch.uint8)
        return flip(codes), flip(exps)

    (kp, ks), (vp, vs) = pool(), pool()
    s = dict(op=c["op"], k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs)
    # the pages of a pool in use lie in any order
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).cpu().numpy()
    table = np.full((B, max_pages), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += int(pages[b])

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)

    s.update(page_table=i32(table), seq_len=i32(p["lens"]), q_start=i32(p["q_start"]) if c["op"] != "decode_q8" else None,
             scale=d ** -0.5, cap=c["cap"], window=c["window"])
    if c["op"].startswith("append"):
        # the projections' fused output: a token's query, key and value heads side by side
        qkv = normal(N, Hq + 2 * Hkv, d)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], interleaved=c["interleaved"], cos_sin=None)
        s["q_start"] = None if int(p["new"].max()) == 1 else s["q_start"]
        s["q_out"] = torch.empty(N, Hq, d, dtype=dt, device=dev)
        s["q_norm"] = (1 + 0.3 * normal(d, dtype=torch.float32)).to(dt) if c["norm"] else None
        s["k_norm"] = (1 + 0.3 * normal(d, dtype=torch.float32)).to(dt) if c["norm"] else None
        s["eps"] = 1e-6
        if c["rot"]:
            half = c["rot"] // 2
            f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
            a = torch.arange(int(p["lens"].max()) + 1, dtype=torch.float64, device=dev)[:, None] * f
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        return s
    # some heads attend sharply, most of them broadly
    sharp = torch.where(torch.arange(Hq, device=dev) % 4 == 3, 1.0, 0.3).to(dt)
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


def _normed(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _rotated(x, cs, interleaved):
    r = cs.shape[1]
    cos, sin = cs[:, None, :r // 2], cs[:, None, r // 2:]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    ab = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([ab, x[..., r:]], -1)


def _append(s):
    v, kp, vp = s["v"], s["k_pages"], s["v_pages"]
    N, B, T = v.shape[0], s["seq_len"].shape[0], kp.shape[1]
    _, seq, _, pos = _rows(s, N, B, v.device)
    q, k = _normed(s["q"], s["q_norm"], s["eps"]), _normed(s["k"], s["k_norm"], s["eps"])
    if s["cos_sin"] is not None:
        cs = s["cos_sin"][pos]
        q, k = _rotated(q, cs, s["interleaved"]), _rotated(k, cs, s["interleaved"])
    page, row = s["page_table"][seq, pos // T].long(), pos % T
    s["q_out"].copy_(q)
    if s["k_scale"] is None:
        kp[page, row] = k.to(kp.dtype)
        vp[page, row] = v
        return s["q_out"], kp, vp
    v = v.float()
    ke, ve = _exponent(k), _exponent(v)
    kp.view(torch.uint8)[page, row] = _codes(k, ke).view(torch.uint8)
    vp.view(torch.uint8)[page, row] = _codes(v, ve).view(torch.uint8)
    s["k_scale"].view(torch.uint8)[page, row] = _e8(ke).view(torch.uint8)
    s["v_scale"].view(torch.uint8)[page, row] = _e8(ve).view(torch.uint8)
    return s["q_out"], kp, vp, s["k_scale"], s["v_scale"]


def _attend(s):
    q, kp, vp, table = s["q"], s["k_pages"], s["v_pages"], s["page_table"]
    N, Hq, d = q.shape
    B, T, Hkv = table.shape[0], kp.shape[1], kp.shape[2]
    G, L = Hq // Hkv, table.shape[1] * T
    start, seq, local, pos = _rows(s, N, B, q.device)
    n = int(N) if B == 1 else int((start[1:] - start[:-1]).max())       # rows of the padded batch
    rows = (start[:-1, None] + torch.arange(n, device=q.device)).clamp(max=N - 1)
    pages = table.clamp(min=0).long()

    def dense(codes, exps):
        x = codes.view(torch.uint8)[pages].view(F8).float() * _two_to(exps.view(torch.uint8)[pages])[..., None]
        return x.reshape(B, L, Hkv, d).transpose(1, 2)

    K, V = dense(kp, s["k_scale"]), dense(vp, s["v_scale"])
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
                       q_out=s["q_out"], cos_sin=s["cos_sin"], interleaved=s["interleaved"], q_start=s["q_start"],
                       q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    if s["op"] == "append_q8":
        E.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_len"], q=s["q"],
                       q_out=s["q_out"], cos_sin=s["cos_sin"], interleaved=s["interleaved"], q_start=s["q_start"],
                       q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"], k_scale=s["k_scale"],
                       v_scale=s["v_scale"])
        return s["q_out"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
    kw = dict(softcap=s["cap"], window=s["window"], slopes=s["slopes"], first_tok=s["first_tok"],
              prefix_len=s["prefix_len"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "decode_q8":
        return E.paged_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_len"], s["scale"], **kw)
    return E.paged_attn_prefill(s["q"], s["q_start"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_len"],
                                s["scale"], **kw)


def run(state):
    if own:
        return _own(state)
    return _append(state) if state["op"].startswith("append") else _attend(state)


# -------------------------------------------------------------- 64-bit definition --
def _e4m3(x):
    """x (float64, |x| <= 448) at the nearest number of four significant bits, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _rows_in_8(x):
    """Codes and numbers 2^e of rows x in float64, by trying the exponents from below."""
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(top.clamp(min=1e-30) / 448)).clamp(-64, 64)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e).clamp(-64, 64)
    return _e4m3((x * torch.exp2(-e)[..., None]).clamp(-448, 448)), torch.exp2(e)


def _values(codes):
    """What e4m3 codes stand for, from their fields."""
    b = codes.view(torch.uint8).long()
    sign, ex, man = 1.0 - 2.0 * (b >> 7), (b >> 3) & 15, (b & 7).double()
    return sign * torch.where(ex > 0, torch.exp2(ex.double() - 7) * (1 + man / 8), man * 2.0 ** -9)


def exact(case, seed):
    c, p, s = case, _plan(case), prepare(case, seed)
    kp, vp, T = s["k_pages"], s["v_pages"], c["page"]
    table = s["page_table"].cpu().numpy()
    if c["op"].startswith("append"):
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        if c["norm"]:
            q = q / (q.pow(2).sum(-1, keepdim=True) / c["d"] + s["eps"]).sqrt() * s["q_norm"].double()
            k = k / (k.pow(2).sum(-1, keepdim=True) / c["d"] + s["eps"]).sqrt() * s["k_norm"].double()
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
        page = torch.from_numpy(table[p["seq"], p["pos"] // T].astype(np.int64)).to(q.device)
        row = torch.from_numpy(p["pos"] % T).to(q.device)
        if c["op"] == "append":
            K, V = kp.double(), vp.double()
            K[page, row], V[page, row] = k, v
            return q, K, V
        K, V = _values(kp), _values(vp)
        ks, vs = (torch.exp2(x.view(torch.uint8).double() - 127) for x in (s["k_scale"], s["v_scale"]))
        K[page, row], ks[page, row] = _rows_in_8(k)
        V[page, row], vs[page, row] = _rows_in_8(v)
        return q, K, V, ks, vs
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
            K, V = (_values(x.view(torch.uint8)[ids, :, h].reshape(-1, d)[:L]) *
                    torch.exp2(e.view(torch.uint8)[ids, :, h].reshape(-1)[:L].double() - 127)[:, None]
                    for x, e in ((kp, s["k_scale"]), (vp, s["v_scale"])))
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
