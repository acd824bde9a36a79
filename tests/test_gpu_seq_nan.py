"""The sequence operators where some values are not finite: what each row and key gets, and that a call takes no longer
than it has to."""
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def p3(cuda_device):
    import geometry_aware_local_b200 as p3
    return p3


def tensors(lq, lk, Hq, Hkv, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(n, h, 64, generator=g, device="cuda").to(dtype)
            for n, h in ((lq, Hq), (lk, Hkv), (lk, Hkv), (lq, Hq))]


def offsets(lens, start=0):
    return torch.tensor([start] + list(start + torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def config(p3, Hq, Hkv, W, S, dtype):
    return p3.make_seq_config(Hq=Hq, Hkv=Hkv, window=W, sinks=S, dtype="bf16" if dtype == torch.bfloat16 else "f32")


def results(p3, cfg, q, k, v, dout, cu_q, cu_k):
    out, lse = p3.window_attn(cfg, q, k, v, cu_q, cu_k)
    return out, lse, *p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,klens,Hq,Hkv,W,S", [
    ([90], [90], 8, 2, 0, 0), ([1], [1], 4, 4, 0, 0), ([333], [333], 8, 1, 40, 3), ([65], [129], 2, 2, 0, 0),
    ([1100], [1100], 8, 2, 0, 0),                # the backward's clusters
    ([40], [3500], 8, 2, 0, 0),                  # the forward's
    ([5000], [5000], 8, 2, 100, 64),             # the narrow tiles, the sinks' pieces
    ([9, 70], [4, 50], 4, 1, 0, 0),
])
def test_rows_behind_a_sequence(p3, cuda_device, lens, klens, Hq, Hkv, W, S, dtype):
    """The tiles reach behind a sequence's end.  What lies there, the next sequence's rows or rows of no sequence, does
    not matter, whatever it is: the same bits as with zeros."""
    nq, nk, more = sum(lens), sum(klens), 70
    cfg = config(p3, Hq, Hkv, W, S, dtype)
    for behind in ([], [more]):                  # rows of no sequence; the next sequence's
        cu_q, cu_k = offsets(lens + behind), offsets(klens + behind)
        got = []
        for value in (0.0, NAN, INF):
            q, k, v, dout = tensors(nq + more, nk + more, Hq, Hkv, dtype)
            q[nq:], k[nk:], v[nk:], dout[nq:] = value, value, value, value
            out, lse, dq, dk, dv = results(p3, cfg, q, k, v, dout, cu_q, cu_k)
            got.append((out[:nq], lse[:nq], dq[:nq], dk[:nk], dv[:nk]))
        for other in got[1:]:
            for a, b in zip(got[0], other):
                assert torch.equal(a, b)


def spread(lens, klens, W, S, q, k, v, dout):
    """Where the results are not finite, from where the inputs are not (NaNs): by the definition, entry by entry."""
    Hq, Hkv = q.shape[1], k.shape[1]
    bad = [~torch.isfinite(t.float()) for t in (q, k, v, dout)]
    out, dq = (torch.zeros_like(bad[0]) for _ in range(2))
    lse = torch.zeros(q.shape[:2], dtype=torch.bool, device=q.device)
    dk, dv = torch.zeros_like(bad[1]), torch.zeros_like(bad[1])
    q0 = k0 = 0
    for lq, lk in zip(lens, klens):
        rq, rk = slice(q0, q0 + lq), slice(k0, k0 + lk)
        ok = ref.visible(lq, lk, W, S, q.device)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            L = (ok & bad[1][rk, g].any(-1)).any(1) | (bad[0][rq, h].any(-1) & ok.any(1))
            o = L[:, None] | (ok.double() @ bad[2][rk, g].double() > 0)
            D = L | (bad[3][rq, h].any(-1) & ok.any(1)) | o.any(-1)
            lse[rq, h], out[rq, h], dq[rq, h] = L, o, D[:, None]
            dk[rk, g] |= (ok & D[:, None]).any(0)[:, None]
            dv[rk, g] |= (ok & L[:, None]).any(0)[:, None] | (ok.double().T @ bad[3][rq, h].double() > 0)
        q0, k0 = q0 + lq, k0 + lk
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


PATTERNS = {
    "v in one dim": lambda q, k, v, d, n: v[n // 2, 0].__setitem__(3, NAN),
    "v in several": lambda q, k, v, d, n: [v[i, -1].__setitem__(i % 64, NAN) for i in range(0, n, 37)],
    "v in a column": lambda q, k, v, d, n: v[:, 0, 11].fill_(NAN),
    "v from a row on": lambda q, k, v, d, n: v[n // 2:].fill_(NAN),
    "k": lambda q, k, v, d, n: k[n // 2, -1].fill_(NAN),
    "q": lambda q, k, v, d, n: q[n // 2].fill_(NAN),
    "dout in one dim": lambda q, k, v, d, n: d[n // 2, 0].__setitem__(5, NAN),
    "dout in several": lambda q, k, v, d, n: [d[i, -1].__setitem__(i % 64, NAN) for i in range(0, n, 41)],
    "dout of the last": lambda q, k, v, d, n: d[n - 1].fill_(NAN),
    "dout everywhere": lambda q, k, v, d, n: d.fill_(NAN),
    "a token": lambda q, k, v, d, n: [t[n // 2].fill_(NAN) for t in (q, k, v, d)],
    "all of v and dout": lambda q, k, v, d, n: [t[:, 0, 9].fill_(NAN) for t in (v, d)],
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("lens,Hq,Hkv,W,S", [([310], 4, 2, 0, 0), ([90, 260], 4, 2, 40, 3), ([700], 8, 1, 150, 64),
                                             ([1100], 2, 2, 0, 0), ([150], 256, 64, 33, 2)],
                         ids=["plain", "windowed", "sinks", "shared", "many heads"])
def test_a_nan_reaches_what_sees_it(p3, cuda_device, lens, Hq, Hkv, W, S, pattern, dtype):
    """Each result is not finite exactly where its definition reads a NaN, dim by dim, and within the tolerance of the
    definition without the NaNs everywhere else."""
    n = sum(lens)
    q, k, v, dout = tensors(n, n, Hq, Hkv, dtype, 3)
    cfg = config(p3, Hq, Hkv, W, S, dtype)
    PATTERNS[pattern](q, k, v, dout, n)
    clean = [torch.nan_to_num(t, nan=0.0) for t in (q, k, v, dout)]
    r = ref.window(*clean[:3], lens, lens, W, S, cfg.softmax_scale, clean[3])
    where = spread(lens, lens, W, S, q, k, v, dout)
    cu = offsets(lens)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), results(p3, cfg, q, k, v, dout, cu, cu)):
        bad = ~torch.isfinite(t.float())
        assert torch.equal(bad, where[name]), (name, int((bad & ~where[name]).sum()), int((~bad & where[name]).sum()))
        ref.close(t[~bad], r[name][~bad], r[name + "_tol"][~bad], name)


@pytest.mark.parametrize("dtype", TYPES)
def test_an_infinity_stays_one_next_to_a_hidden_nan(p3, cuda_device, dtype):
    """Infinities that a row or a key sees are its result, whatever NaNs lie near that it does not see."""
    n, a, b = 300, 130, 170
    q, k, v, dout = tensors(n, n, 2, 1, dtype, 4)
    cfg, cu = config(p3, 2, 1, 0, 0, dtype), offsets([n])
    v[a, 0, 5], v[b, 0, 5] = INF, NAN
    dout[b, :, 7], dout[a, :, 7] = INF, NAN
    out, lse, dq, dk, dv = results(p3, cfg, q, k, v, dout, cu, cu)
    assert torch.isfinite(out[:a].float()).all()
    assert (out[a:b, :, 5] == INF).all() and torch.isnan(out[b:, :, 5]).all()
    assert torch.isfinite(out[:, :, 6].float()).all()
    assert torch.isnan(dv[:a + 1, :, 7]).all() and (dv[a + 1:b + 1, :, 7] == INF).all()
    assert torch.isfinite(dv[b + 1:].float()).all() and torch.isfinite(dv[:, :, 8].float()).all()
    # a row whose delta is infinite, without a NaN anywhere: dv does not read it
    q, k, v, dout = tensors(n, n, 2, 1, dtype, 4)
    dout[b, 0, 7] = INF
    out, lse, dq, dk, dv = results(p3, cfg, q, k, v, dout, cu, cu)
    assert (dv[:b + 1, 0, 7] == INF).all() and torch.isfinite(dv[:, :, :7].float()).all()
    assert torch.isfinite(dv[b + 1:].float()).all() and torch.isfinite(dk[b + 1:].float()).all()
    assert not torch.isfinite(dk[:b + 1].float()).any() and not torch.isfinite(dq[b, 0].float()).any()


def test_a_scale_so_small_that_the_terms_overflow(p3, cuda_device):
    """lse / scale, which the key side subtracts from the products, is beyond a float: equal weights all the same."""
    n = 200
    q, k, v, dout = tensors(n, n, 2, 1, torch.bfloat16, 4)
    for W, S in ((0, 0), (50, 3)):
        cfg, cu = config(p3, 2, 1, W, S, torch.bfloat16), offsets([n])
        cfg.softmax_scale = 2.0 ** -125
        r = ref.window(q, k, v, [n], [n], W, S, cfg.softmax_scale, dout)
        for name, t in zip(("out", "lse", "dq", "dk", "dv"), results(p3, cfg, q, k, v, dout, cu, cu)):
            ref.close(t, r[name], r[name + "_tol"], name)


def milliseconds(f):
    best = INF
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 8192), (torch.float32, 2048)])
def test_a_nan_costs_little(p3, cuda_device, dtype, n):
    """Without a window, where a NaN reaches up to every row: results that have to be NaN are not formed again from
    all that they see (which took 50 to 800 times as long as the call), and what a hidden NaN has spoilt are a tile's
    rows at most."""
    cfg, cu = config(p3, 8, 2, 0, 0, dtype), offsets([n])
    half = n // 2 + 14

    def both(change):
        q, k, v, dout = tensors(n, n, 8, 2, dtype, 8)
        change(q, k, v, dout)
        out, lse = p3.window_attn(cfg, q, k, v, cu)
        p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
        return (milliseconds(lambda: p3.window_attn(cfg, q, k, v, cu)),
                milliseconds(lambda: p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)))

    clean = both(lambda q, k, v, d: None)
    for limit, change in (
            (5, lambda q, k, v, d: v[0, :, 3].fill_(NAN)), (5, lambda q, k, v, d: k[0].fill_(NAN)),
            (5, lambda q, k, v, d: q[n - 1].fill_(NAN)), (5, lambda q, k, v, d: d[n - 1].fill_(NAN)),
            (5, lambda q, k, v, d: d.fill_(NAN)), (5, lambda q, k, v, d: d[:, :, 7].fill_(NAN)),
            (5, lambda q, k, v, d: v[:, 0, 7].fill_(NAN)),
            (45, lambda q, k, v, d: v[half:].fill_(NAN)), (45, lambda q, k, v, d: d[half].fill_(NAN)),
            (45, lambda q, k, v, d: [t[half].fill_(NAN) for t in (q, k, v, d)])):
        got = both(change)
        assert got[0] <= limit * clean[0] and got[1] <= limit * clean[1], (limit, got, clean)
