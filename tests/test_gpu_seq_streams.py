"""The causal sequence operators as part of a program: streams, CUDA graphs, the bounded waits' error path, calls that
overlap, and the binding's refusals."""
import math

import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu

LIMIT_US = 2000


@pytest.fixture(scope="module")
def p3(cuda_device):
    import geometry_aware_local_b200 as p3
    return p3


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def tensors(lq, lk, Hq, Hkv, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(n, h, 64, generator=g, device="cuda").to(dtype)
            for n, h in ((lq, Hq), (lk, Hkv), (lk, Hkv), (lq, Hq))]


# ---- few query tiles before many keys: the forward's cluster path ---------------------

@pytest.mark.parametrize("lens,klens,Hq,Hkv,W,S", [
    ([70, 3], [4000, 2500], 8, 2, 0, 0), ([70, 3], [4000, 2500], 8, 2, 1500, 10), ([1], [3500], 2, 1, 0, 0),
    ([300], [2111], 4, 4, 0, 0), ([5, 0, 64], [1700, 30, 1], 8, 1, 0, 0), ([40, 40], [10, 3300], 4, 1, 0, 0),
])
def test_few_queries_before_many_keys(p3, lens, klens, Hq, Hkv, W, S):
    q, k, v, dout = tensors(sum(lens), sum(klens), Hq, Hkv)
    cfg = p3.make_seq_config(Hq=Hq, Hkv=Hkv, window=W, sinks=S)
    cu_q, cu_k = offsets(lens), offsets(klens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = p3.window_attn(cfg, q, k, v, cu_q, cu_k, err=err)
    grads = p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
    assert p3.check_status(err) == 0
    r = ref.window(q, k, v, lens, klens, W, S, cfg.softmax_scale, dout)
    ref.close(out, r["out"], r["out_tol"], "out")
    ref.close(lse, r["lse"], r["lse_tol"], "lse")
    for n, g in zip(("dq", "dk", "dv"), grads):
        ref.close(g, r[n], r[n + "_tol"], n)


def test_hidden_nan_in_a_shared_tile(p3):
    """The cluster path computes a row again whose product with a hidden value was not a number."""
    lens, klens, W = [40], [3500], 1200
    q, k, v, _ = tensors(40, 3500, 8, 2)
    cfg = p3.make_seq_config(window=W)
    r = ref.window(q, k, v, lens, klens, W, 0, cfg.softmax_scale)
    k[3490], v[3490] = float("nan"), float("inf")        # seen from row 30 on
    v[2262] = float("nan")                               # seen by the rows 0 and 1 only
    out, lse = p3.window_attn(cfg, q, k, v, offsets(lens), offsets(klens))
    clean = slice(2, 30)
    ref.close(out[clean], r["out"][clean], r["out_tol"][clean], "out")
    ref.close(lse[clean], r["lse"][clean], r["lse_tol"][clean], "lse")
    assert torch.isnan(out[:2].float()).all() and torch.isnan(out[30:].float()).all()


@pytest.mark.parametrize("lens,klens,Hq,Hkv,W,S", [
    ([1100], [1100], 8, 2, 0, 0), ([900, 1, 300], [900, 1, 300], 4, 1, 700, 5), ([130], [700], 8, 1, 0, 0),
    ([2100], [2100], 8, 1, 100, 64), ([700], [650], 2, 1, 0, 0), ([1500], [1500], 1, 1, 300, 2),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_of_few_tiles(p3, lens, klens, Hq, Hkv, W, S, dtype):
    """The CTAs of a cluster share a tile's steps in the backward, some of them without one."""
    q, k, v, dout = (t.to(dtype) for t in tensors(sum(lens), sum(klens), Hq, Hkv))
    cfg = p3.make_seq_config(Hq=Hq, Hkv=Hkv, window=W, sinks=S, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    cu_q, cu_k = offsets(lens), offsets(klens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = p3.window_attn(cfg, q, k, v, cu_q, cu_k, err=err)
    grads = p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
    again = p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
    assert p3.check_status(err) == 0
    r = ref.window(q, k, v, lens, klens, W, S, cfg.softmax_scale, dout)
    ref.close(out, r["out"], r["out_tol"], "out")
    for n, a, b in zip(("dq", "dk", "dv"), grads, again):
        ref.close(a, r[n], r[n + "_tol"], n)
        assert torch.equal(a, b)


# ---- bounded waits -----------------------------------------------------------------------

@pytest.mark.parametrize("lens,klens,W,S", [([5], [5], 0, 0), ([700], [700], 100, 4), ([70], [4000], 0, 0),
                                              ([5000], [5000], 100, 4)],
                         ids=["one-tile", "several", "cluster", "narrow"])
def test_times_out_then_recovers(p3, lens, klens, W, S):
    """Every tensor-core kernel withholds its last tile: the call reports the timeout, and the same call without the
    flag is right afterwards.  (The waits are bounded at 2 ms; nothing faults or hangs.)"""
    q, k, v, dout = tensors(sum(lens), sum(klens), 8, 2)
    cu_q, cu_k = offsets(lens), offsets(klens)
    cfg = p3.make_seq_config(window=W, sinks=S)
    bad = p3.make_seq_config(window=W, sinks=S, flags=p3.FLAG_DIAG_STALL, wait_limit_us=LIMIT_US)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = p3.window_attn(cfg, q, k, v, cu_q, cu_k, err=err)
    grads = p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
    assert p3.check_status(err) == 0
    p3.window_attn(bad, q, k, v, cu_q, cu_k, err=err)
    assert p3.check_status(err) == 8
    p3.window_attn_bwd(bad, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
    assert p3.check_status(err) == 8
    again, again_lse = p3.window_attn(cfg, q, k, v, cu_q, cu_k, err=err)
    more = p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
    assert p3.check_status(err) == 0
    assert torch.equal(again, out) and torch.equal(again_lse, lse)
    for a, b in zip(more, grads):
        assert torch.equal(a, b)


# ---- streams ----------------------------------------------------------------------------------

def test_calls_follow_the_work_on_their_stream(p3):
    """Inputs replaced on a side stream right before each call, several calls behind one another on one workspace."""
    lens = [900, 77]
    cfg = p3.make_seq_config(window=200, sinks=3)
    cu = offsets(lens)
    sets = [tensors(977, 977, 8, 2, seed=s) for s in (1, 2)]
    want = []
    for q, k, v, d in sets:
        out, lse = p3.window_attn(cfg, q, k, v, cu)
        want.append([out, lse, *p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, d)])
    torch.cuda.synchronize()
    buf = [torch.empty_like(t) for t in sets[0]]
    ws = torch.empty(p3.window_attn_bwd_workspace_bytes(cfg, 2, 977, 977), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    outs = [[torch.empty_like(t) for t in want[0]] for _ in range(4)]
    for i in range(4):
        with torch.cuda.stream(side):
            for b, t in zip(buf, sets[i % 2]):
                b.copy_(t)
        o = outs[i]
        p3.window_attn(cfg, *buf[:3], cu, out=o[0], lse=o[1], stream=side)      # not the current stream
        p3.window_attn_bwd(cfg, *buf[:3], cu, None, o[0], o[1], buf[3], *o[2:], workspace=ws, stream=side.cuda_stream)
        got.append(o)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        for a, b in zip(o, want[i % 2]):
            assert torch.equal(a, b)


def test_an_explicit_stream_needs_the_callers_memory(p3):
    q, k, v, d = tensors(32, 32, 8, 2)
    cfg, cu, s = p3.make_seq_config(window=8), offsets([32]), torch.cuda.Stream()
    out, lse = p3.window_attn(cfg, q, k, v, cu)
    pages = torch.zeros(2, 64, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, n = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for call in (lambda: p3.window_attn(cfg, q, k, v, cu, stream=s),
                 lambda: p3.window_attn_bwd(cfg, q, k, v, cu, cu, out, lse, d, stream=s),
                 lambda: p3.cache_attn(cfg, q[:1], pages, pages, table, n, stream=s),
                 lambda: p3.cache_evict(cfg, pages, pages, table, n, torch.zeros(1, 64, device="cuda"), table, 1, 0,
                                        stream=s)):
        with pytest.raises(ValueError, match="explicit stream"):
            call()


def test_refusals_on_the_device(p3):
    """Strided, short, wrongly typed and half-given tensors."""
    q, k, v, d = tensors(32, 32, 8, 2)
    cfg, cu = p3.make_seq_config(window=8), offsets([32])
    out, lse = p3.window_attn(cfg, q, k, v, cu)
    for call, match in (
            (lambda: p3.window_attn(cfg, q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cu), "contiguous"),
            (lambda: p3.window_attn(cfg, q, k[:16], v, cu), "shape"),
            (lambda: p3.window_attn(cfg, q, k, v.float(), cu), "must be"),
            (lambda: p3.window_attn(cfg, q, k, v, cu.long()), "must be"),
            (lambda: p3.window_attn(cfg, q, k, v, cu, cu[:1]), "shape"),
            (lambda: p3.window_attn(cfg, q, k, v, cu, out=out), "both"),
            (lambda: p3.window_attn_bwd(cfg, q, k, v, cu, cu, out, lse, d, dq=q), "all of"),
            (lambda: p3.window_attn(cfg, q, k, v, cu, err=torch.zeros(1, device="cuda")), "error word"),
            (lambda: p3.window_attn_bwd(cfg, q, k, v, cu, cu, out, lse, d,
                                        workspace=torch.empty(8, dtype=torch.uint8)), "workspace")):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(p3.Pack3DError, match="WORKSPACE"):
        p3.window_attn_bwd(cfg, q, k, v, cu, cu, out, lse, d,
                           workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_no_sequence_at_all(p3):
    cfg, cu = p3.make_seq_config(window=8), torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v, d = tensors(6, 4, 8, 2)
    out, lse = p3.window_attn(cfg, q, k, v, cu)
    assert (out == 0).all() and (lse == -math.inf).all()
    for g in p3.window_attn_bwd(cfg, q, k, v, cu, cu, out, lse, d):
        assert (g == 0).all()
    for rows in ((0, 4), (4, 0), (0, 0)):
        q, k, v, d = tensors(*rows, 8, 2)
        for dtype, name in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
            c = p3.make_seq_config(window=8, dtype=name)
            a = [t.to(dtype) for t in (q, k, v, d)]
            cu_q, cu_k = offsets([rows[0]]), offsets([rows[1]])
            out, lse = p3.window_attn(c, *a[:3], cu_q, cu_k)
            assert (out == 0).all() and (lse == -math.inf).all()
            for g in p3.window_attn_bwd(c, *a[:3], cu_q, cu_k, out, lse, a[3]):
                assert (g == 0).all()


# ---- CUDA graphs ---------------------------------------------------------------------------------

def test_captured_and_replayed(p3):
    """One decoding step (append, attention with weights, an eviction) and one training step, captured and replayed on
    new inputs of other lengths; two graphs with their own workspaces replayed at the same time."""
    dev = torch.device("cuda")
    cfg = p3.make_seq_config(Hq=8, Hkv=2, sinks=2, page=16)
    cache = p3.PagedCache(cfg, 3, 2048, budget=64)
    k, v = (torch.randn(1700, 2, 64, device=dev).bfloat16() for _ in range(2))
    cache.append(k, v, offsets([1500, 30, 170]))
    q1, k1, v1 = (torch.randn(3, h, 64, device=dev).bfloat16() for h in (8, 2, 2))
    cfg_w = p3.make_seq_config(window=50, sinks=1)
    q, kk, vv, d = tensors(300, 300, 8, 2)
    cu = offsets([200, 100])
    leaves = [t.requires_grad_(True) for t in (q, kk, vv)]

    def decode():
        p3.cache_append(cfg, k1, v1, cache.k_pages, cache.v_pages, cache.table, cache.lengths, err=cache.err)
        n = cache.lengths + 1
        w = torch.zeros_like(cache.weights)
        out, lse = p3.cache_attn(cfg, q1, cache.k_pages, cache.v_pages, cache.table, n, weights=w, err=cache.err)
        return out, lse, w, *p3.cache_evict(cfg, cache.k_pages, cache.v_pages, cache.table, n, w, cache.spare, 64, 8,
                                            err=cache.err)

    def train():
        out = p3.window_attention(cfg_w, *leaves, cu)
        return (out, *torch.autograd.grad(out, leaves, d))

    graphs = []
    for step in (decode, train):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step()
        graphs.append((g, res, step, s))
    with torch.no_grad():
        for t in (q1, k1, v1, q, kk, vv, d):
            t.copy_(torch.randn_like(t))
        cache.lengths.copy_(torch.tensor([77, 900, 0], device=dev))
        cache.k_pages.normal_()
        cache.v_pages.normal_()
        cu.copy_(torch.tensor([0, 13, 290], device=dev))
    torch.cuda.synchronize()
    for g, _, _, s in graphs:
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    for g, res, step, _ in graphs:
        want = step()
        inside = torch.ones_like(res[0], dtype=torch.bool)
        for a, b in zip(res, want):
            assert torch.equal(a, b)
    cache.check()


def test_two_streams_at_once(p3):
    """The same operator on two streams with buffers of their own, many calls in flight."""
    cfg = p3.make_seq_config(window=64, sinks=2, page=16)
    sets = [tensors(1500, 1500, 8, 2, seed=s) for s in (5, 6)]
    cu = offsets([1000, 500])
    caches = []
    for q, k, v, _ in sets:
        c = p3.PagedCache(cfg, 2, 1600)
        c.append(k, v, cu)
        caches.append(c)
    calls = [lambda i=i: (*p3.window_attn(cfg, *sets[i][:3], cu), caches[i].attend(sets[i][0][:2].contiguous()))
             for i in (0, 1)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for i in (0, 1):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)
