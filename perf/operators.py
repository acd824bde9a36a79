"""The causal sequence operators and their paged key-value cache, as a user's program calls them: their cases, plain
forms, least work and values in 64 bits.

Five passes are measured.  "window": causal attention with a sliding window and a few first tokens that stay visible,
over packed sequences of different lengths.  "grad": the same forward and the gradients of q, k and v.  "append": new
keys and values into a paged cache.  "decode": attention of one new token per sequence over that cache.  "evict": the
cache cut to a budget by accumulated attention weight.

With ``own`` false ``run`` computes the plain form in elementary torch operations, in 32 bits, rounded once at the end;
with ``own`` true it calls the operators of geometry_aware_local_b200.
"""
import math

import numpy as np
import torch

own = False

DH = 64          # head dim of every operator of the framework
BAND = 128       # queries that share one band of keys in the plain windowed form


def _case(op, name=None, **values):
    c = {"op": op, "dtype": "bf16", "Hq": 8, "Hkv": 2, "window": 0, "sinks": 0}
    c.update(values)
    if name is not None:
        c["name"] = name
    return c


def _ragged(rng, batch, longest):
    """`batch` lengths spread over the logarithm of 1 .. longest, the longest among them."""
    got = [max(1, int(longest ** rng.random())) for _ in range(batch - 1)] + [longest]
    rng.shuffle(got)
    return ",".join(str(n) for n in got)


def listed():
    import random
    r = random.Random(11)
    return [
        # a few short prompts packed together before the model answers: the launch is most of the time
        _case("window", "window short prompts", lens="7,130,1,63", window=128, sinks=4),
        # one volume's 65,536 tokens read as one sequence with a local window (the benchmark's heads and token count)
        _case("window", "window 64k", lens="65536", window=1024, sinks=4),
        # the last 2,048 tokens of a long prompt that is taken in piece by piece; eight heads share one key head
        _case("window", "window chunk of 16k", lens="2048", klens="16384", Hq=8, Hkv=1),
        # a training step over packed documents
        _case("grad", "grad packed 16k", lens="9000,5001,2383", window=512, sinks=4),
        # the float form, which is used to check models, at odd sizes
        _case("grad", "grad float", lens="1500,1,549", window=200, sinks=1, Hq=4, Hkv=2, dtype="f32"),
        # one new token for each of 64 sequences
        _case("append", "append step", lens=",".join(["1"] * 64), old=_ragged(r, 64, 4000), page=64),
        # the prompts of a batch written into the cache at once
        _case("append", "append prompts", lens="32768,20011,9001,3757", old="0,5,640,17", page=64),
        # one new token of one short chat
        _case("decode", "decode one", old="311", page=64, capacity=512),
        # a served batch of very different lengths
        _case("decode", "decode ragged", old=",".join(str(r.randint(1, 32768)) for _ in range(48)), page=64,
              capacity=32768),
        # a float cache whose attention weights are wanted, for the eviction below
        _case("decode", "decode float weights", old="4096,1,777,2049,3000,64,65,12,1500", page=32, capacity=4096,
              dtype="f32", Hq=4, Hkv=4, weights=True),
        # one long chat cut to a small cache
        _case("evict", "evict one", old="1400", page=64, capacity=1536, budget=1024, recent=128, sinks=4),
        # a batch of long chats, all cut at once
        _case("evict", "evict batch", old=",".join(str(6000 + 137 * i) for i in range(16)), page=64, capacity=8192,
              budget=4096, recent=512, sinks=4),
    ]


def draw(rng):
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))  # noqa: E731
    op = rng.choice(("window", "window", "grad", "grad", "append", "decode", "decode", "evict"))
    G = rng.choice((1, 2, 4, 8))
    Hkv = rng.choice([h for h in (1, 2, 3, 4, 8) if h * G <= 16])
    f32 = rng.random() < 0.25
    heads = {"Hq": G * Hkv, "Hkv": Hkv, "dtype": "f32" if f32 else "bf16"}
    if op in ("window", "grad"):
        most = 3000 if f32 else (40000 if op == "window" else 16000)
        if rng.random() < 0.3:       # no window: every earlier token; keys may be more than queries
            total = log(8, min(most, 6000) * 2 // max(2, Hkv * G // 4))
            cuts = sorted(rng.randint(0, total) for _ in range(rng.randint(0, 3)))
            lens = [max(1, b - a) for a, b in zip([0] + cuts, cuts + [total])]
            klens = [n + (int(total * rng.random() / 4) if rng.random() < 0.5 else 0) for n in lens]
            return _case(op, lens=",".join(map(str, lens)), klens=",".join(map(str, klens)), **heads)
        window = log(16, 300 if f32 else 2048)
        total = log(50, max(60, int(most * 8 / max(8, Hkv * G) * min(1.0, 1024 / window))))
        lens = _ragged(rng, rng.randint(1, 6), total)
        return _case(op, lens=lens, window=window, sinks=rng.choice((0, 1, 4, rng.randint(0, 64))), **heads)
    page = rng.choice((16, 32, 64, 128))
    batch = log(1, 48)
    if op == "append":
        lens = _ragged(rng, batch, 1 if rng.random() < 0.4 else log(2, 40000 // Hkv))
        return _case(op, lens=lens, old=_ragged(rng, batch, log(1, 4000)), page=page, **heads)
    if op == "decode":
        longest = log(16, min(32768, 2 * 64 * 32768 // (batch * Hkv * (2 if f32 else 1)) // 2))
        windowed = rng.random() < 0.3
        return _case(op, old=_ragged(rng, batch, longest), page=page, capacity=-(-longest // page) * page,
                     weights=rng.random() < 0.4, window=log(16, longest) if windowed else 0,
                     sinks=rng.randint(0, 8) if windowed else 0, **heads)
    longest = log(200, 8000)
    budget = max(64, int(longest * rng.uniform(0.2, 0.9)))
    sinks = rng.randint(0, 8)
    return _case(op, old=_ragged(rng, min(batch, 16), longest), page=page, capacity=-(-longest // page) * page,
                 budget=budget, recent=rng.randint(0, budget - sinks), **dict(heads, sinks=sinks))


# ---- inputs ---------------------------------------------------------------------

def _ints(text):
    return [int(x) for x in text.split(",")]


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pages(n, page):
    return -(-n // page)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)
    host = np.random.RandomState(int(seed) % (2 ** 31))
    dt, op, Hq, Hkv = _type(case), case["op"], case["Hq"], case["Hkv"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def offsets(lens):
        return ints([0] + list(np.cumsum(lens)))

    s = {"case": case}
    if op in ("window", "grad"):
        lens = _ints(case["lens"])
        klens = _ints(case.get("klens", case["lens"]))
        s["q"] = normal(sum(lens), Hq, DH)
        s["k"], s["v"] = normal(sum(klens), Hkv, DH), normal(sum(klens), Hkv, DH)
        s["cu_q"] = offsets(lens)
        s["cu_k"] = s["cu_q"] if lens == klens else offsets(klens)
        s["same"] = lens == klens
        if op == "grad":
            s["dout"] = normal(sum(lens), Hq, DH)
        return s
    page, old = case["page"], _ints(case["old"])
    batch = len(old)
    if op == "append":
        lens = _ints(case["lens"])
        wide = max(_pages(a + b, page) for a, b in zip(old, lens))
        s["k"], s["v"] = normal(sum(lens), Hkv, DH), normal(sum(lens), Hkv, DH)
        s["cu"] = offsets(lens)
        pages = sum(_pages(a + b, page) for a, b in zip(old, lens))
        need = [_pages(a + b, page) for a, b in zip(old, lens)]
    else:
        wide = case["capacity"] // page
        need = [_pages(a, page) for a in old]
        pages = sum(need)
    spare = _pages(case["budget"], page) * batch if op == "evict" else 0
    order = host.permutation(pages + spare).astype(np.int32)
    table = np.zeros((batch, wide), np.int32)
    at = 0
    for b in range(batch):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"] = torch.from_numpy(table).to(dev)
    s["lengths"] = ints(old)
    s["k_pages"] = normal(pages + spare, page, Hkv, DH)
    s["v_pages"] = normal(pages + spare, page, Hkv, DH)
    if op == "decode":
        s["q"] = normal(batch, Hq, DH)
        if case.get("weights"):
            s["weights"] = torch.zeros(batch, case["capacity"], device=dev)
    if op == "evict":
        # accumulated weights: a few tokens carry most of it, and equal values occur
        w = torch.exp(2 * torch.randn(batch, case["capacity"], generator=gen, device=dev))
        s["weights"] = torch.floor(w * 64) / 64
        s["new_table"] = torch.from_numpy(order[pages:].reshape(batch, -1).copy()).to(dev)
    return s


# ---- the operators -----------------------------------------------------------------

def _config(s):
    """The configuration that a program makes once and keeps."""
    import geometry_aware_local_b200 as p3
    if "cfg" not in s:
        c = s["case"]
        s["cfg"] = p3.make_seq_config(Hq=c["Hq"], Hkv=c["Hkv"], window=c["window"], sinks=c["sinks"],
                                      page=c.get("page", 64), dtype=c["dtype"])
    return p3, s["cfg"]


def run(s):
    op = s["case"]["op"]
    if op == "window":
        return _window_own(s) if own else _window_plain(s, s["q"], s["k"], s["v"])
    if op == "grad":
        return _grad(s)
    if op == "append":
        return _append_own(s) if own else _append_plain(s)
    if op == "decode":
        return _decode_own(s) if own else _decode_plain(s)
    return _evict_own(s) if own else _evict_plain(s)


def _window_own(s):
    p3, cfg = _config(s)
    out, lse = p3.window_attn(cfg, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
    return {"out": out, "lse": lse}


def _grad(s):
    q, k, v = (s[n].detach().requires_grad_(True) for n in ("q", "k", "v"))
    if own:
        p3, cfg = _config(s)
        out = p3.window_attention(cfg, q, k, v, s["cu_q"], s["cu_k"])
    else:
        out = _window_plain(s, q, k, v)["out"]
    dq, dk, dv = torch.autograd.grad(out, (q, k, v), s["dout"])
    return {"out": out.detach(), "dq": dq, "dk": dk, "dv": dv}


def _append_own(s):
    p3, cfg = _config(s)
    p3.cache_append(cfg, s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["cu"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _decode_own(s):
    p3, cfg = _config(s)
    out, lse = p3.cache_attn(cfg, s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"],
                             weights=s.get("weights"))
    r = {"out": out, "lse": lse}
    if "weights" in s:
        r["weights"] = s["weights"]
    return r


def _evict_own(s):
    p3, cfg = _config(s)
    kept, weights, lengths = p3.cache_evict(cfg, s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["weights"],
                                            s["new_table"], s["case"]["budget"], s["case"]["recent"])
    return {"kept": kept, "weights": weights, "lengths": lengths, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ---- their plain forms ---------------------------------------------------------------

def _rows(cu, total):
    """The sequence of every packed row, and its place in it."""
    at = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), at, right=True)
    return seq, at - cu[seq].long()


def _softmax(x):
    """Softmax along the last axis and its log-sum-exp, for rows of which some or all values are -inf."""
    top = x.amax(-1, keepdim=True).detach()
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    return p, (top + torch.log(total)).squeeze(-1)


def _window_plain(s, q, k, v):
    c = s["case"]
    Hkv, G, W, S = c["Hkv"], c["Hq"] // c["Hkv"], c["window"], c["sinks"]
    Tq, Tk, scale = q.shape[0], k.shape[0], 1 / math.sqrt(DH)
    qf, kf, vf = q.float().view(Tq, Hkv, G, DH), k.float(), v.float()
    qseq, at = _rows(s["cu_q"], Tq)
    lq, lk = (torch.diff(cu).long() for cu in (s["cu_q"], s["cu_k"]))
    pos = at + (lk - lq)[qseq]                         # a query's place among its sequence's keys
    if W == 0 or not s["same"] or Tk <= 2 * (W + BAND):
        kseq, kat = _rows(s["cu_k"], Tk)
        ahead = pos[:, None] - kat[None]
        see = (qseq[:, None] == kseq[None]) & (ahead >= 0)
        if W:
            see &= (ahead < W) | (kat[None] < S)
        x = torch.einsum("qhgd,khd->hgqk", qf, kf) * scale
        p, lse = _softmax(x.masked_fill(~see, -math.inf))
        out = torch.einsum("hgqk,khd->qhgd", p, vf)
        return {"out": out.reshape(q.shape).to(q.dtype), "lse": lse.permute(2, 0, 1).reshape(Tq, -1)}
    # Bands: BAND consecutive queries against the W + BAND - 1 keys that end with them, and the first S keys apart.
    n = _pages(Tq, BAND)
    pad = n * BAND - Tq
    grow = torch.nn.functional.pad
    qb = grow(qf, (0, 0, 0, 0, 0, 0, 0, pad)).view(n, BAND, Hkv, G, DH)
    kb, vb = (grow(x, (0, 0, 0, 0, W - 1, pad)).unfold(0, W + BAND - 1, BAND) for x in (kf, vf))
    posb, seqb = (grow(x, (0, pad), value=-1).view(n, BAND) for x in (pos, qseq))
    kpos, kseq = (grow(x, (W - 1, pad), value=-2).unfold(0, W + BAND - 1, BAND) for x in (pos, qseq))
    ahead = posb[:, :, None] - kpos[:, None]
    see = (seqb[:, :, None] == kseq[:, None]) & (ahead >= 0) & (ahead < W)
    x = torch.einsum("nqhgd,nhdk->nhgqk", qb, kb) * scale
    x = x.masked_fill(~see[:, None, None], -math.inf)
    first = s["cu_k"].long()[qseq][:, None] + torch.arange(S, device=q.device)
    far = pos[:, None] - torch.arange(S, device=q.device) >= W
    first = torch.where(far, first, torch.zeros_like(first))
    y = (qf[:, None] * kf[first][:, :, :, None]).sum(-1) * scale                       # [Tq, S, Hkv, G]
    y = y.masked_fill(~far[:, :, None, None], -math.inf)
    yb = grow(y, (0, 0, 0, 0, 0, 0, 0, pad), value=-math.inf).view(n, BAND, S, Hkv, G).permute(0, 3, 4, 1, 2)
    p, lse = _softmax(torch.cat((x, yb), -1))
    out = torch.einsum("nhgqk,nhdk->nqhgd", p[..., :W + BAND - 1], vb).reshape(n * BAND, Hkv, G, DH)[:Tq]
    ps = p[..., W + BAND - 1:].permute(0, 3, 4, 1, 2).reshape(n * BAND, S, Hkv, G)[:Tq]
    out = out + (ps[..., None] * vf[first][:, :, :, None]).sum(1)
    lse = lse.permute(0, 3, 1, 2).reshape(n * BAND, Hkv * G)[:Tq]
    return {"out": out.reshape(q.shape).to(q.dtype), "lse": lse}


def _slots(s, at):
    """Rows of the page pool (pages x page) of the slots `at` [batch, n] of every sequence."""
    page = s["case"]["page"]
    return s["table"].long().gather(1, at // page) * page + at % page


def _append_plain(s):
    seq, at = _rows(s["cu"], s["k"].shape[0])
    to = s["lengths"].long()[seq] + at
    page = s["case"]["page"]
    row = s["table"].long()[seq, to // page] * page + to % page
    s["k_pages"].view(-1, *s["k"].shape[1:])[row] = s["k"]
    s["v_pages"].view(-1, *s["v"].shape[1:])[row] = s["v"]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _decode_plain(s):
    c = s["case"]
    Hkv, G, cap = c["Hkv"], c["Hq"] // c["Hkv"], c["capacity"]
    batch = s["q"].shape[0]
    at = torch.arange(cap, device=s["q"].device)[None]
    n = s["lengths"].long()[:, None]
    see = at < n
    if c["window"]:
        see = see & ((n - 1 - at < c["window"]) | (at < c["sinks"]))
    row = _slots(s, at.expand(batch, cap))
    k = s["k_pages"].view(-1, Hkv, DH)[row].float()
    v = s["v_pages"].view(-1, Hkv, DH)[row].float()
    x = torch.einsum("bhgd,bkhd->bhgk", s["q"].float().view(batch, Hkv, G, DH), k) / math.sqrt(DH)
    p, lse = _softmax(x.masked_fill(~see[:, None, None], -math.inf))
    out = torch.einsum("bhgk,bkhd->bhgd", p, v)
    r = {"out": out.reshape(s["q"].shape).to(s["q"].dtype), "lse": lse.reshape(batch, -1)}
    if "weights" in s:
        s["weights"].copy_(torch.where(at < n, p.sum((1, 2)), s["weights"]))
        r["weights"] = s["weights"]
    return r


def _evict_plain(s):
    c = s["case"]
    budget, batch = c["budget"], s["table"].shape[0]
    at = torch.arange(c["capacity"], device=s["table"].device)[None]
    n = s["lengths"].long()[:, None]
    stay = (at < c["sinks"]) | (at >= n - c["recent"])
    rank = torch.where(at < n, torch.where(stay, math.inf, s["weights"]), -math.inf)
    best = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :budget]
    if best.shape[1] < budget:
        best = torch.nn.functional.pad(best, (0, budget - best.shape[1]), value=c["capacity"])
    best = torch.sort(torch.where(best < n, best, c["capacity"]), dim=1).values
    have = best < n
    kept = torch.where(have, best, -1)
    src = _slots(s, torch.where(have, best, 0))
    page = c["page"]
    to = torch.arange(budget, device=best.device)
    dst = s["new_table"].long()[:, to // page] * page + to % page
    for_all = have[:, :, None, None]
    k, v = (s[m].view(-1, c["Hkv"], DH) for m in ("k_pages", "v_pages"))
    k[dst] = torch.where(for_all, k[src], k[dst])
    v[dst] = torch.where(for_all, v[src], v[dst])
    w = torch.zeros(batch, s["new_table"].shape[1] * page, device=best.device)
    w[:, :budget] = torch.where(have, s["weights"].gather(1, torch.where(have, best, 0)), 0.0)
    return {"kept": kept.int(), "weights": w, "lengths": have.sum(1).int(), "k_pages": s["k_pages"],
            "v_pages": s["v_pages"]}


# ---- least work ------------------------------------------------------------------------

def _pairs(case):
    """Visible (query, key) pairs of one head."""
    W, S = case["window"], case["sinks"]
    total = 0
    for n, m in zip(_ints(case["lens"]), _ints(case.get("klens", case["lens"]))):
        pos = np.arange(m - n, m, dtype=np.int64)
        seen = np.maximum(pos + 1, 0)
        if W:
            near = np.minimum(seen, W)
            seen = near + np.minimum(seen - near, S)
        total += int(seen.sum())
    return total


def work(case):
    op, Hq, Hkv = case["op"], case["Hq"], case["Hkv"]
    eb = 2 if case["dtype"] == "bf16" else 4
    if op in ("window", "grad"):
        tq, tk = sum(_ints(case["lens"])), sum(_ints(case.get("klens", case["lens"])))
        qb, kb = tq * Hq * DH * eb, tk * Hkv * DH * eb
        flops = 4 * DH * Hq * _pairs(case)
        if op == "window":
            return {"bytes": 2 * qb + 2 * kb + 4 * tq * Hq, "flops": flops}
        # backward: the scores again, dP, and three products with dS and P; q, k, v, dout in, out and three gradients out
        return {"bytes": 4 * qb + 4 * kb, "flops": flops + 10 * DH * Hq * _pairs(case)}
    row = 2 * Hkv * DH * eb
    if op == "append":
        return {"bytes": 2 * row * sum(_ints(case["lens"])), "flops": 0}
    old = _ints(case["old"])
    if op == "decode":
        W = case["window"]
        seen = sum(n if not W else min(n, W) + min(max(0, n - W), case["sinks"]) for n in old)
        extra = 4 * sum(old) if case.get("weights") else 0
        return {"bytes": row * seen + 2 * len(old) * Hq * DH * eb + extra, "flops": 4 * DH * Hq * seen}
    rows = sum(min(n, case["budget"]) for n in old)
    return {"bytes": 2 * row * rows + 4 * sum(old) + 8 * rows, "flops": 0}


# ---- values in 64 bits --------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("window", "grad"):
        return _exact_window(case, s)
    if op == "append":
        return _exact_append(case, s)
    if op == "decode":
        return _exact_decode(case, s)
    return _exact_evict(case, s)


def _exact_window(case, s):
    """Sequence by sequence, head by head, a block of queries at a time."""
    W, S, Hq, G = case["window"], case["sinks"], case["Hq"], case["Hq"] // case["Hkv"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    grad = case["op"] == "grad"
    if grad:
        do, dq, dk, dv = s["dout"].double(), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    q0 = k0 = 0
    for n, m in zip(_ints(case["lens"]), _ints(case.get("klens", case["lens"]))):
        block = 512
        for a in range(0, n, block):
            z = min(n, a + block)
            i = torch.arange(a, z, device=q.device) + (m - n)
            last = z - 1 + m - n
            if last < 0:
                continue
            low = max(0, a + m - n - W + 1) if W else 0
            j = torch.arange(low, last + 1, device=q.device)
            if W and S and low > 0:
                j = torch.cat((torch.arange(0, min(S, low), device=q.device), j))
            ok = j[None] <= i[:, None]
            if W:
                ok &= (i[:, None] - j[None] < W) | (j[None] < S)
            rows, cols = slice(q0 + a, q0 + z), k0 + j
            for h in range(Hq):
                g = h // G
                kk, vv, qq = k[cols, g], v[cols, g], q[rows, h]
                t = (qq @ kk.T / 8.0).masked_fill(~ok, -math.inf)
                e = torch.logsumexp(t, 1)
                p = torch.nan_to_num(torch.exp(t - e[:, None]), nan=0.0)
                lse[rows, h] = e
                out[rows, h] = p @ vv
                if grad:
                    d = do[rows, h]
                    ds = p * (d @ vv.T - (d * out[rows, h]).sum(1, keepdim=True))
                    dq[rows, h] = ds @ kk / 8.0
                    dk[:, g].index_add_(0, cols, ds.T @ qq / 8.0)
                    dv[:, g].index_add_(0, cols, p.T @ d)
        q0, k0 = q0 + n, k0 + m
    if grad:
        return {"out": out, "dq": dq, "dk": dk, "dv": dv}
    return {"out": out, "lse": lse}


def _exact_append(case, s):
    k, v = s["k_pages"].clone(), s["v_pages"].clone()
    page, at = case["page"], 0
    table = s["table"].cpu().numpy()
    for b, (n, start) in enumerate(zip(_ints(case["lens"]), _ints(case["old"]))):
        slot = np.arange(start, start + n)
        where = torch.from_numpy(table[b, slot // page].astype(np.int64)).to(k.device)
        inside = torch.from_numpy(slot % page).to(k.device)
        k[where, inside], v[where, inside] = s["k"][at:at + n], s["v"][at:at + n]
        at += n
    return {"k_pages": k.double(), "v_pages": v.double()}


def _exact_decode(case, s):
    page, G, W = case["page"], case["Hq"] // case["Hkv"], case["window"]
    q = s["q"].double()
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    weights = s["weights"].double() if "weights" in s else None
    for b, n in enumerate(_ints(case["old"])):
        ids = s["table"][b, :_pages(n, page)].long()
        k, v = (s[m][ids].reshape(-1, case["Hkv"], DH)[:n].double() for m in ("k_pages", "v_pages"))
        j = torch.arange(n, device=q.device)
        hide = torch.zeros(n, dtype=torch.bool, device=q.device)
        if W:
            hide = (n - 1 - j >= W) & (j >= case["sinks"])
        total = torch.zeros(n, dtype=torch.float64, device=q.device)
        for h in range(case["Hq"]):
            t = (k[:, h // G] @ q[b, h] / 8.0).masked_fill(hide, -math.inf)
            lse[b, h] = torch.logsumexp(t, 0)
            p = torch.exp(t - lse[b, h])
            out[b, h] = p @ v[:, h // G]
            total += p
        if weights is not None:
            weights[b, :n] = total
    r = {"out": out, "lse": lse}
    if weights is not None:
        r["weights"] = weights
    return r


def _exact_evict(case, s):
    page, budget = case["page"], case["budget"]
    k, v = s["k_pages"].clone(), s["v_pages"].clone()
    table, new = s["table"].cpu().numpy().astype(np.int64), s["new_table"].cpu().numpy().astype(np.int64)
    w = s["weights"].cpu().numpy()
    batch = len(table)
    kept = np.full((batch, budget), -1, np.int64)
    weights = np.zeros((batch, new.shape[1] * page))
    lengths = np.zeros(batch, np.int64)
    for b, n in enumerate(_ints(case["old"])):
        keep = np.arange(n)
        if n > budget:
            head, tail = np.arange(case["sinks"]), np.arange(n - case["recent"], n)
            middle = np.arange(case["sinks"], n - case["recent"])
            order = np.lexsort((middle, -w[b, middle].astype(np.float64)))
            keep = np.sort(np.concatenate((head, tail, middle[order[:budget - len(head) - len(tail)]])))
        m = len(keep)
        lengths[b], kept[b, :m], weights[b, :m] = m, keep, w[b, keep]
        to = np.arange(m)
        src, dst = (torch.from_numpy(x).to(k.device) for x in (table[b, keep // page], new[b, to // page]))
        si, di = (torch.from_numpy(x).to(k.device) for x in (keep % page, to % page))
        k[dst, di], v[dst, di] = s["k_pages"][src, si], s["v_pages"][src, si]
    whole = lambda x: torch.from_numpy(x).to(s["k_pages"].device)  # noqa: E731
    return {"kept": whole(kept).int(), "weights": whole(weights), "lengths": whole(lengths).int(),
            "k_pages": k.double(), "v_pages": v.double()}
