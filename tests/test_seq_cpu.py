"""The causal sequence operators without a GPU: configs, sizes and refusals of the C ABI and the binding, and the
64-bit reference of their GPU tests against autograd and differences."""
import ctypes
import math

import pytest
import torch

import seq_reference as ref


@pytest.fixture(scope="module")
def p3():
    import geometry_aware_local_b200 as p3
    return p3


def test_default_config(p3):
    c = p3.SeqConfig()
    p3.lib.pack3d_default_seq_config(ctypes.byref(c))
    assert (c.Hq, c.Hkv, c.d_h, c.dtype, c.window, c.sinks, c.page) == (8, 2, 64, p3.BF16, 0, 0, 64)
    assert abs(c.softmax_scale - 0.125) < 1e-9
    assert p3.validate_seq(c) == 0
    assert p3.validate_seq(p3.make_seq_config()) == 0
    assert ctypes.sizeof(p3.SeqConfig) == 48


@pytest.mark.parametrize("field,value,status", [
    ("d_h", 128, 2), ("Hq", 6, 2), ("Hq", 0, 2), ("Hkv", 3, 2), ("Hq", 32, 2), ("Hkv", -2, 2), ("dtype", 7, 4),
    ("softmax_scale", 0.0, 1), ("softmax_scale", math.inf, 1), ("softmax_scale", math.nan, 1), ("window", -1, 1),
    ("sinks", -1, 2), ("sinks", 65, 2), ("page", 0, 2), ("page", 8, 2), ("page", 48, 2), ("page", 512, 2),
    ("flags", 0x10, 1), ("wait_limit_us", -1, 1), ("reserved0", 1, 1), ("reserved1", 1, 1),
])
def test_validate_rejects(p3, field, value, status):
    c = p3.make_seq_config()
    setattr(c, field, value)
    assert p3.validate_seq(c) == status
    cp, L, fake = ctypes.byref(c), p3.lib, 1 << 20
    assert L.pack3d_window_attn(cp, 1, 8, 8, *[fake] * 6, fake, 0, None, None) == status
    assert L.pack3d_cache_attn_workspace_bytes(cp, 1, 1, 0) == 0
    assert L.pack3d_window_attn_bwd_workspace_bytes(cp, 1, 8, 8) == 0


@pytest.mark.parametrize("field,value", [("window", 2 ** 31 - 1), ("sinks", 64), ("page", 16), ("page", 256),
                                         ("flags", 0x8), ("wait_limit_us", 1), ("Hq", 2), ("Hq", 16)])
def test_validate_accepts(p3, field, value):
    c = p3.make_seq_config()
    setattr(c, field, value)
    assert p3.validate_seq(c) == 0


def test_window_refusals(p3):
    """Counts, null and misaligned pointers and a small workspace are refused before anything is launched."""
    c, L, fake = p3.make_seq_config(window=16), p3.lib, 1 << 20
    cp, bad16, bad4 = ctypes.byref(c), fake + 8, fake + 2

    def fwd(batch=1, tq=8, tk=8, cu_q=fake, cu_k=fake, q=fake, k=fake, v=fake, out=fake, lse=fake):
        return L.pack3d_window_attn(cp, batch, tq, tk, cu_q, cu_k, q, k, v, out, lse, 0, None, None)

    assert fwd(batch=0) == 0 and fwd(tq=0) == 0
    assert fwd(batch=-1) == 1 and fwd(tq=-1) == 1 and fwd(tk=-1) == 1
    assert fwd(batch=65536) == 2 and fwd(tq=1 << 24) == 2 and fwd(tk=1 << 24) == 2
    for name in ("cu_q", "cu_k", "q", "k", "v", "out"):
        assert fwd(**{name: None}) == 1, name
    for name in ("q", "k", "v", "out"):
        assert fwd(**{name: bad16}) == 3, name
    for name in ("cu_q", "cu_k", "lse"):
        assert fwd(**{name: bad4}) == 3, name

    need = p3.window_attn_bwd_workspace_bytes(c, 1, 8, 8)
    assert need >= 8 * 8 * 4

    def bwd(batch=1, tq=8, tk=8, ws=fake, size=need, **kw):
        a = dict.fromkeys(("cu_q", "cu_k", "q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"), fake)
        a.update(kw)
        return L.pack3d_window_attn_bwd(cp, batch, tq, tk, *a.values(), 0, ws, size, None, None)

    assert bwd(batch=0) == 0 and bwd(tq=0, tk=0) == 0 and bwd(batch=-1) == 1 and bwd(tq=1 << 24) == 2
    for name in ("cu_q", "cu_k", "q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"):
        assert bwd(**{name: None}) == 1, name
        assert bwd(**{name: bad4 if name in ("cu_q", "cu_k", "lse") else bad16}) == 3, name
    assert bwd(ws=None) == 6 and bwd(ws=fake + 16) == 6 and bwd(size=need - 1) == 6


def test_cache_refusals(p3):
    c, L, fake = p3.make_seq_config(sinks=4), p3.lib, 1 << 20
    cp, bad16, bad4 = ctypes.byref(c), fake + 8, fake + 2

    def append(batch=2, rows=2, cu=None, max_pages=4, num_pages=8, **kw):
        a = dict.fromkeys(("lengths", "table", "k", "v", "k_pages", "v_pages"), fake)
        a.update(kw)
        return L.pack3d_cache_append(cp, batch, rows, cu, a["lengths"], a["table"], max_pages, num_pages, a["k"],
                                     a["v"], a["k_pages"], a["v_pages"], None, None)

    assert append(batch=0, rows=0) == 0 and append(rows=0, cu=fake) == 0
    assert append(rows=3) == 1 and append(batch=-1) == 1 and append(max_pages=-1) == 1 and append(num_pages=-1) == 1
    assert append(rows=-1, cu=fake) == 1 and append(rows=1 << 24, cu=fake) == 2
    assert append(batch=65536, rows=65536) == 2 and append(max_pages=1 << 25) == 2 and append(num_pages=1 << 25) == 2
    for name in ("lengths", "table", "k", "v", "k_pages", "v_pages"):
        assert append(**{name: None}) == 1, name
        assert append(**{name: bad4 if name in ("lengths", "table") else bad16}) == 3, name

    need = p3.cache_attn_workspace_bytes(c, 2, 4, True)
    assert need > 0 == p3.cache_attn_workspace_bytes(c, 2, 4, False)      # short, no weights: none needed
    assert p3.cache_attn_workspace_bytes(c, 2, 400, False) > 0

    def attn(batch=2, ws=fake, size=need, max_pages=4, num_pages=8, **kw):
        a = dict.fromkeys(("q", "k_pages", "v_pages", "table", "lengths", "out", "lse", "weights"), fake)
        a.update(kw)
        return L.pack3d_cache_attn(cp, batch, a["q"], a["k_pages"], a["v_pages"], a["table"], max_pages, num_pages,
                                   a["lengths"], a["out"], a["lse"], a["weights"], 0, ws, size, None, None)

    assert attn(batch=0) == 0 and attn(batch=-1) == 1 and attn(batch=65536) == 2 and attn(max_pages=1 << 25) == 2
    for name in ("q", "k_pages", "v_pages", "table", "lengths", "out"):
        assert attn(**{name: None}) == 1, name
    for name in ("q", "k_pages", "v_pages", "out"):
        assert attn(**{name: bad16}) == 3, name
    for name in ("table", "lengths", "lse", "weights"):
        assert attn(**{name: bad4}) == 3, name
    assert attn(ws=None) == 6 and attn(ws=fake + 16) == 6 and attn(size=need - 1) == 6

    def evict(batch=2, budget=64, recent=8, max_pages=4, num_pages=8, new_max=1, **kw):
        names = ("k_pages", "v_pages", "table", "lengths", "weights", "new_table", "kept", "new_weights",
                 "new_lengths")
        a = dict.fromkeys(names, fake)
        a.update(kw)
        return L.pack3d_cache_evict(cp, batch, a["k_pages"], a["v_pages"], num_pages, a["table"], max_pages,
                                    a["lengths"], a["weights"], budget, recent, a["new_table"], new_max, a["kept"],
                                    a["new_weights"], a["new_lengths"], None, None)

    assert evict(batch=0) == 0
    assert evict(budget=0) == 1 and evict(budget=65) == 1 and evict(recent=61) == 1 and evict(recent=-1) == 1
    assert evict(batch=-1) == 1 and evict(new_max=-1) == 1 and evict(new_max=1 << 25) == 2
    for name in ("k_pages", "v_pages", "table", "lengths", "weights", "new_table", "kept", "new_weights",
                 "new_lengths"):
        assert evict(**{name: None}) == 1, name
        assert evict(**{name: bad16 if name in ("k_pages", "v_pages") else bad4}) == 3, name


def test_outputs_over_inputs_are_refused(p3):
    """A result that lies over an input, or over another result, by its first or its last byte: refused, since other
    parts of the call still read there.  (Every call here is refused: the addresses are of nothing.)"""
    c, L = p3.make_seq_config(window=16, page=16), p3.lib
    cp, gap = ctypes.byref(c), 1 << 24

    def each(call, names, sizes, outputs, allowed=()):
        at = {n: gap * (i + 1) for i, n in enumerate(names)}
        for a in outputs:
            for b in names:
                if a == b or (a, b) in allowed:
                    continue
                for where in (at[b], at[b] + sizes[b] - 16 if sizes[b] > 16 else at[b], at[b] - sizes[a] + 16):
                    if where % 256 and a == "workspace":
                        continue
                    assert call(**dict(at, **{a: where})) == 1, (a, b, where - at[b])

    tq, tk, row_q, row_k = 96, 80, 8 * 128, 2 * 128
    sizes = {"q": tq * row_q, "k": tk * row_k, "v": tk * row_k, "out": tq * row_q, "lse": tq * 32, "cu_q": 16, "cu_k": 16,
             "dout": tq * row_q, "dq": tq * row_q, "dk": tk * row_k, "dv": tk * row_k}
    sizes["workspace"] = need = p3.window_attn_bwd_workspace_bytes(c, 3, tq, tk)
    each(lambda **a: L.pack3d_window_attn(cp, 3, tq, tk, *a.values(), 0, None, None),
         ("cu_q", "cu_k", "q", "k", "v", "out", "lse"), sizes, ("out", "lse"))
    each(lambda workspace, **a: L.pack3d_window_attn_bwd(cp, 3, tq, tk, *a.values(), 0, workspace, need, None, None),
         ("cu_q", "cu_k", "q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "workspace"), sizes,
         ("dq", "dk", "dv", "workspace"))

    batch, wide, pages = 4, 8, 40
    sizes = {"q": batch * row_q, "out": batch * row_q, "lse": batch * 32, "k_pages": pages * 16 * row_k,
             "v_pages": pages * 16 * row_k, "table": batch * wide * 4, "lengths": batch * 4, "weights": batch * wide * 64,
             "kept": batch * 256, "new_table": batch * 16, "new_weights": batch * 4 * 64, "new_lengths": batch * 4}
    sizes["workspace"] = need = p3.cache_attn_workspace_bytes(c, batch, wide, True)
    each(lambda q, k_pages, v_pages, table, lengths, out, lse, weights, workspace:
         L.pack3d_cache_attn(cp, batch, q, k_pages, v_pages, table, wide, pages, lengths, out, lse, weights, 0, workspace,
                             need, None, None),
         ("q", "k_pages", "v_pages", "table", "lengths", "out", "lse", "weights", "workspace"),
         sizes, ("lse", "weights", "workspace"))
    each(lambda q, k_pages, v_pages, table, lengths, out, lse, weights, workspace:
         L.pack3d_cache_attn(cp, batch, q, k_pages, v_pages, table, wide, pages, lengths, out, lse, weights, 0, workspace,
                             need, None, None),
         ("q", "k_pages", "v_pages", "table", "lengths", "out", "lse", "weights", "workspace"),
         sizes, ("out",), allowed=(("out", "q"),))
    each(lambda k_pages, v_pages, table, lengths, weights, new_table, kept, new_weights, new_lengths:
         L.pack3d_cache_evict(cp, batch, k_pages, v_pages, pages, table, wide, lengths, weights, 64, 8, new_table, 4, kept,
                              new_weights, new_lengths, None, None),
         ("k_pages", "v_pages", "table", "lengths", "weights", "new_table", "kept", "new_weights", "new_lengths"),
         sizes, ("kept", "new_weights", "new_lengths"),
         allowed=[(a, b) for a in ("kept", "new_weights", "new_lengths") for b in ("k_pages", "v_pages")])


def test_status_texts(p3):
    assert p3.STATUS[9] == "LENGTHS" and p3.STATUS[10] == "PAGE"
    for st in (9, 10):
        assert p3._status_string(st) not in ("ok", "unknown status")


def test_binding_refuses_cpu_tensors_and_wrong_types(p3):
    c = p3.make_seq_config()
    q, k = torch.zeros(4, 8, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        p3.window_attn(c, q, k, k, cu)
    with pytest.raises(ValueError, match="q must be torch.bfloat16"):
        p3.window_attn(c, q.float(), k, k, cu)
    with pytest.raises(ValueError, match="shape"):
        p3.window_attn(c, q[:, :4], k, k, cu)
    with pytest.raises(p3.Pack3DError, match="SHAPE"):
        p3.window_attn(p3.make_seq_config(d_h=128), q, k, k, cu)
    pages = torch.zeros(4, 64, 2, 64, dtype=torch.bfloat16)
    table, lengths = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        p3.cache_attn(c, q[:1], pages, pages, table, lengths)
    with pytest.raises(ValueError, match="shape"):
        p3.cache_append(c, k, k, pages[:, :32], pages[:, :32], table, lengths)
    with pytest.raises(ValueError, match="capacity"):
        p3.PagedCache(c, 1, 64, budget=65)


def test_cache_refuses_another_kind_of_device(p3):
    for device in ("cpu", "meta"):
        with pytest.raises(ValueError, match="CUDA device"):
            p3.PagedCache(p3.make_seq_config(), 1, 64, device=device)


# ---- the reference itself ------------------------------------------------------------

def test_reference_masks():
    """Against the definition, entry by entry."""
    for lq, lk, W, S in ((5, 5, 2, 1), (3, 9, 4, 2), (4, 2, 0, 0), (1, 7, 1, 3)):
        ok = ref.visible(lq, lk, W, S)
        for r in range(lq):
            p = lk - lq + r
            for j in range(lk):
                assert bool(ok[r, j]) == (0 <= j <= p and (W == 0 or p - j < W or j < S))


def test_reference_gradients():
    """The reference's gradients against autograd of its forward, and against central differences."""
    g = torch.Generator().manual_seed(3)
    lens, klens, W, S, scale = [5, 3], [7, 3], 3, 1, 0.125
    q = torch.randn(8, 4, 64, generator=g)
    k, v = torch.randn(10, 2, 64, generator=g), torch.randn(10, 2, 64, generator=g)
    dout = torch.randn(8, 4, 64, generator=g)
    r = ref.window(q, k, v, lens, klens, W, S, scale, dout)

    def loss(q, k, v):
        total, q0, k0 = 0.0, 0, 0
        for lq, lk in zip(lens, klens):
            ok = ref.visible(lq, lk, W, S)
            for h in range(4):
                x = q[q0:q0 + lq, h] @ k[k0:k0 + lk, h // 2].T * scale
                p = torch.softmax(x.masked_fill(~ok, -math.inf), -1)
                total = total + (dout[q0:q0 + lq, h].double() * (p @ v[k0:k0 + lk, h // 2])).sum()
            q0, k0 = q0 + lq, k0 + lk
        return total

    leaves = [t.double().requires_grad_(True) for t in (q, k, v)]
    auto = torch.autograd.grad(loss(*leaves), leaves)
    for n, t in zip(("dq", "dk", "dv"), auto):
        assert torch.allclose(r[n], t, rtol=1e-9, atol=1e-12), n
    plain = [t.detach() for t in leaves]
    for which, name in enumerate(("dq", "dk", "dv")):
        for at in ((0, 0, 0), (2, 1, 17), (6, 1, 63)):
            step = 1e-5
            ends = []
            for s in (step, -step):
                moved = [t.clone() for t in plain]
                moved[which][at] += s
                ends.append(float(loss(*moved)))
            assert abs((ends[0] - ends[1]) / (2 * step) - float(r[name][at])) < 1e-7
