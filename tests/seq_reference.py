"""The causal sequence operators from their definition in 64 bits, with the sums that the tests' tolerances are made
of.  Plain torch on whatever device the inputs are on; no code of the package."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative to the value


def visible(lq, lk, window, sinks, device="cpu"):
    p = torch.arange(lk - lq, lk, device=device)[:, None]
    j = torch.arange(lk, device=device)[None]
    ok = j <= p
    if window:
        ok &= (p - j < window) | (j < sinks)
    return ok


def softmax_rows(x, ok):
    """Softmax over the visible entries of each row and its log-sum-exp: 0 and -inf for a row that sees nothing."""
    x = x.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.where(ok, torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None]),
                    torch.zeros_like(x))
    return p, lse


def window(q, k, v, lens, klens, W, S, scale, dout=None):
    """Values, and how far a kernel may be off: its sums are in 32 bits, its probabilities and score gradients are
    rounded to the operands' type once (bf16) before the products, its results once at the end.

    With u half a step of the type, f = 2^-24 and n terms in a sum, for each row
      score      |ds| <= f (66) scale sum_d |q_d k_d|                         (64 products, the sum, the scale)
      probability |dp| <= p (u + 2 ds + 8 f + n f)                            (rounding, both scores, exp, the sum)
      out        |do| <= sum_j |dp_j| |v_j| + n f sum p|v| + u |o|
    and the same bookkeeping for the gradients.  The bf16 kernels round P to bf16 (u), the float ones do not, but u is
    2^-24 there and is left in."""
    u, f = U[q.dtype], 2.0 ** -24
    G = q.shape[1] // k.shape[1]
    qd, kd, vd = (t.double() for t in (q, k, v))
    r = {"out": torch.zeros_like(qd), "out_tol": torch.zeros_like(qd)}
    r["lse"] = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    r["lse_tol"] = torch.zeros_like(r["lse"])
    if dout is not None:
        dd = dout.double()
        for n, t in (("dq", qd), ("dk", kd), ("dv", vd)):
            r[n], r[n + "_tol"] = torch.zeros_like(t), torch.zeros_like(t)
    q0 = k0 = 0
    for lq, lk in zip(lens, klens):
        ok = visible(lq, lk, W, S, q.device)
        for h in range(q.shape[1]):
            g = h // G
            rq, rk = slice(q0, q0 + lq), slice(k0, k0 + lk)
            # What is hidden from every query never enters the reference's products either.
            Q, K, V = qd[rq, h], kd[rk, g], vd[rk, g]
            Qa, Ka, Va = Q.abs(), K.abs(), V.abs()
            p, lse = softmax_rows(Q @ K.T * scale, ok)
            ds = 66 * f * scale * (Qa @ Ka.T)
            worst = torch.where(ok, ds, torch.zeros_like(ds)).amax(1, keepdim=True) if lk else ds.new_zeros(lq, 1)
            terms = ok.sum(1, keepdim=True)
            rel = ds + worst + (8 + terms) * f
            dp = p * (u + rel)
            o = p @ V
            A = p @ Va
            otol = dp @ Va + terms * f * A + u * o.abs()
            r["out"][rq, h], r["out_tol"][rq, h] = o, otol
            r["lse"][rq, h] = lse
            # the scores, the sum, and the logarithm's and the result's own steps
            r["lse_tol"][rq, h] = (worst + (8 + terms) * f).squeeze(1) + 4 * f * torch.nan_to_num(lse.abs(), posinf=0)
            if dout is None:
                continue
            D = dd[rq, h]
            Da = D.abs()
            t = D @ V.T
            delta = (D * o).sum(1, keepdim=True)
            dS = p * (t - delta)
            # <dout, v> and <dout, out> are sums of 64 products; out comes with its own error
            dt = 66 * f * (Da @ Va.T)
            ddelta = (Da * otol).sum(1, keepdim=True) + 66 * f * (Da * o.abs()).sum(1, keepdim=True)
            ddS = dS.abs() * (u + rel) + p * (1 + rel) * (dt + ddelta)
            r["dq"][rq, h] = scale * (dS @ K)
            r["dq_tol"][rq, h] = scale * (ddS @ Ka + (terms + 2) * f * (dS.abs() @ Ka)) + u * r["dq"][rq, h].abs()
            many = ok.sum(0)[:, None] * G
            r["dk"][rk, g] += scale * (dS.T @ Q)
            r["dk_tol"][rk, g] += scale * (ddS.T @ Qa + (many + 2) * f * (dS.abs().T @ Qa))
            r["dv"][rk, g] += p.T @ D
            r["dv_tol"][rk, g] += dp.T @ Da + many * f * (p.T @ Da)
        q0, k0 = q0 + lq, k0 + lk
    if dout is not None:
        for n in ("dk", "dv"):
            r[n + "_tol"] += u * r[n].abs()
    return r


def decode(q, k_pages, v_pages, table, lengths, W, S, scale):
    """One new token per sequence over the paged cache, as window() of one query per sequence, and the weights."""
    B, page = table.shape[0], k_pages.shape[1]
    rows_k, rows_v = [], []
    for b in range(B):
        n = int(lengths[b])
        ids = table[b, :-(-n // page)].long()
        rows_k.append(k_pages[ids].reshape(-1, *k_pages.shape[2:])[:n])
        rows_v.append(v_pages[ids].reshape(-1, *v_pages.shape[2:])[:n])
    lens, klens = [1] * B, [int(n) for n in lengths]
    k, v = torch.cat(rows_k), torch.cat(rows_v)
    r = window(q, k, v, lens, klens, W, S, scale)
    weights = torch.zeros(B, table.shape[1] * page, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(weights)
    f, G = 2.0 ** -24, q.shape[1] // k_pages.shape[2]
    for b, n in enumerate(klens):
        if n == 0:
            continue
        ok = visible(1, n, W, S, q.device)
        for h in range(q.shape[1]):
            K = rows_k[b][:, h // G].double()
            Q = q[b:b + 1, h].double()
            p, _ = softmax_rows(Q @ K.T * scale, ok)
            ds = 66 * f * scale * (Q.abs() @ K.abs().T)
            weights[b, :n] += p[0]
            tol[b, :n] += (p * (ds + ds.amax() + (16 + n + q.shape[1]) * f))[0]
    r["weights"], r["weights_tol"] = weights, tol
    return r


def evict(lengths, weights, budget, sinks, recent):
    """Old slots that stay, per sequence, in order."""
    kept = []
    for b, n in enumerate(int(x) for x in lengths):
        if n <= budget:
            kept.append(list(range(n)))
            continue
        w = [float(x) + 0.0 for x in weights[b]]
        rank = sorted(range(sinks, n - recent), key=lambda j: (0, -w[j], j) if w[j] == w[j] else (1, 0.0, j))
        stay = rank[:budget - sinks - recent]
        kept.append(sorted(list(range(sinks)) + stay + list(range(n - recent, n))))
    return kept


def close(got, want, tol, what=""):
    """Every value within its own tolerance; infinities equal."""
    got = got.double()
    same = got == want
    off = (got - want).abs()
    bad = ~(same | (off <= tol + 1e-30))
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: got "
                             f"{float(got[tuple(i)])}, want {float(want[tuple(i)])} within {float(tol[tuple(i)]):.3g}")
