"""The causal sequence operators on the GPU against their definition in 64 bits (seq_reference.py), at the sizes and
masks where they can go wrong."""
import random

import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def p3(cuda_device):
    import geometry_aware_local_b200 as p3
    return p3


def offsets(lens, dev):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=dev)


def inputs(lens, klens, Hq, Hkv, dtype, dev, seed=0, pad=0):
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(rows, heads):
        return torch.randn(rows, heads, 64, generator=g, device=dev).to(dtype)

    q, dout = normal(sum(lens) + pad, Hq), normal(sum(lens) + pad, Hq)
    return q, normal(sum(klens) + pad, Hkv), normal(sum(klens) + pad, Hkv), dout


def check_window(p3, lens, klens, Hq, Hkv, W, S, dtype, dev, seed=0):
    q, k, v, dout = inputs(lens, klens, Hq, Hkv, dtype, dev, seed)
    cfg = p3.make_seq_config(Hq=Hq, Hkv=Hkv, window=W, sinks=S, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    cu_q, cu_k = offsets(lens, dev), offsets(klens, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = p3.window_attn(cfg, q, k, v, cu_q, cu_k, err=err)
    dq, dk, dv = p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
    assert p3.check_status(err) == 0
    r = ref.window(q, k, v, lens, klens, W if W else 0, S, cfg.softmax_scale, dout)
    ref.close(out, r["out"], r["out_tol"], "out")
    ref.close(lse, r["lse"], r["lse_tol"], "lse")
    ref.close(dq, r["dq"], r["dq_tol"], "dq")
    ref.close(dk, r["dk"], r["dk_tol"], "dk")
    ref.close(dv, r["dv"], r["dv_tol"], "dv")


TYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,klens,Hq,Hkv,W,S", [
    ([1], [1], 8, 2, 0, 0),                       # one token
    ([2, 1, 3], [2, 1, 3], 1, 1, 1, 0),           # a window of the token itself
    ([63], [63], 4, 1, 0, 0), ([64], [64], 4, 4, 16, 2), ([65], [65], 2, 1, 33, 64),
    ([127, 1, 129], [127, 1, 129], 8, 2, 50, 4),
    ([500], [500], 8, 1, 100, 64),                # eight heads share a key head; as many sinks as there can be
    ([300, 0, 211], [300, 0, 211], 6, 3, 97, 1),  # an empty sequence between others; three key heads
    ([700], [700], 2, 2, 0, 7),                   # sinks without a window change nothing
    ([33, 5], [400, 260], 8, 2, 0, 0),            # the last queries of longer sequences
    ([40, 130], [700, 130], 4, 2, 64, 3),
    ([9, 70], [4, 50], 4, 1, 0, 0),               # more queries than keys: the first see nothing
    ([5, 3], [0, 3], 2, 1, 8, 1),                 # no key at all
    ([200], [200], 1, 1, 2 ** 31 - 1, 0),         # a window longer than anything
    ([1000], [1000], 2, 1, 96, 5), ([513], [513], 16, 2, 511, 0), ([450], [450], 8, 8, 128, 0),
])
def test_window_and_gradients(p3, cuda_device, lens, klens, Hq, Hkv, W, S, dtype):
    check_window(p3, lens, klens, Hq, Hkv, W, S, dtype, cuda_device)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,W,S", [([9000, 1200], 700, 5), ([8300, 1, 40], 0, 0)])
def test_long_sequences(p3, cuda_device, lens, W, S, dtype):
    check_window(p3, lens, lens, 2, 1, W, S, dtype, cuda_device)


def test_many_sequences(p3, cuda_device):
    """More sequences than one pass over the offsets takes at once, most of them short."""
    lens = [(7 * i) % 23 for i in range(150)]
    check_window(p3, lens, lens, 4, 1, 9, 2, torch.bfloat16, cuda_device)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,W,S", [(2, 1, 20, 3), (8, 1, 0, 0)])
def test_hundreds_of_sequences(p3, cuda_device, Hq, Hkv, W, S, dtype):
    """Two steps of the search for a CTA's sequence; empty ones, ones of one token and ones of several tiles among
    them, and keys of their own lengths."""
    r = random.Random(5)
    lens = [r.choice((0, 1, 1, 2, 9, 31, 33)) for _ in range(230)] + [300, 0, 1] + [r.choice((0, 5)) for _ in range(60)]
    klens = [n + r.choice((0, 0, 3, 130)) for n in lens]
    check_window(p3, lens, klens, Hq, Hkv, W, S, dtype, cuda_device)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,klens,Hq,Hkv,W,S", [
    ([65], [65], 320, 320, 33, 64),                    # every key a sink
    ([300], [300], 240, 120, 33, 64),                  # two tiles of sinks
    ([300, 0, 211], [300, 0, 211], 120, 120, 97, 1),
    ([40, 130], [700, 130], 640, 160, 64, 3),
    ([9, 70], [4, 50], 400, 200, 0, 0),                # more queries than keys
    ([1], [1], 1024, 1024, 0, 0),
    ([500], [500], 1024, 128, 100, 64),
    ([31, 32, 33], [64, 96, 160], 400, 200, 32, 33),
])
def test_as_many_heads_as_fill_the_gpu(p3, cuda_device, lens, klens, Hq, Hkv, W, S, dtype):
    """Enough tiles for the narrow key tiles of the bf16 forward, and for a CTA a tile in float, at the masks' edges."""
    check_window(p3, lens, klens, Hq, Hkv, W, S, dtype, cuda_device)


def test_hidden_nan_in_narrow_tiles(p3, cuda_device):
    dev, n, W, S, bad = cuda_device, 5000, 40, 3, 2500
    q, k, v, _ = inputs([n], [n], 8, 2, torch.bfloat16, dev, 7)
    cfg = p3.make_seq_config(window=W, sinks=S)
    r = ref.window(q, k, v, [n], [n], W, S, cfg.softmax_scale)
    v[bad], k[bad] = float("nan"), float("inf")
    out, lse = p3.window_attn(cfg, q, k, v, offsets([n], dev))
    rows = torch.arange(n, device=dev)
    reads = (rows >= bad) & (rows - bad < W)
    assert torch.isnan(out[reads].float()).all()
    ref.close(out[~reads], r["out"][~reads], r["out_tol"][~reads], "out")
    ref.close(lse[~reads], r["lse"][~reads], r["lse_tol"][~reads], "lse")


def test_as_many_sequences_as_there_may_be(p3, cuda_device):
    """Sequences of one token: the softmax of one score is 1, so out is v, and dv the group's dout."""
    dev, n = cuda_device, 65535
    q, k, v, dout = inputs([n], [n], 2, 1, torch.bfloat16, dev, 3)
    cfg = p3.make_seq_config(Hq=2, Hkv=1, window=16, sinks=1)
    cu = torch.arange(n + 1, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = p3.window_attn(cfg, q, k, v, cu, err=err)
    dv = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout, err=err)[2]
    assert p3.check_status(err) == 0
    assert torch.equal(out, v.expand(-1, 2, -1))
    score = (q.double() * k.double()).sum(-1) / 8
    assert ((lse.double() - score).abs() <= 2.0 ** -24 * (66 * (q.double() * k.double()).abs().sum(-1) / 8
                                                          + 16 + 4 * score.abs())).all()
    # P is within 2^-20 of 1 and rounds to 1; the sum of two and its rounding are left
    want = dout.double().sum(1, keepdim=True)
    assert ((dv.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs() + 2.0 ** -23 * dout.double().abs().sum(
        1, keepdim=True)).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_values_of_every_size(p3, cuda_device, dtype):
    """Large scores (one key takes all the weight) and equal scores."""
    dev = cuda_device
    q, k, v, dout = inputs([300], [300], 4, 2, dtype, dev, 5)
    cfg = p3.make_seq_config(Hq=4, Hkv=2, window=77, sinks=2, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    cu = offsets([300], dev)
    for scale in (0.0, 12.0):
        qs = (q.float() * scale).to(dtype)
        out, lse = p3.window_attn(cfg, qs, k, v, cu)
        grads = p3.window_attn_bwd(cfg, qs, k, v, cu, None, out, lse, dout)
        r = ref.window(qs, k, v, [300], [300], 77, 2, cfg.softmax_scale, dout)
        ref.close(out, r["out"], r["out_tol"], "out")
        ref.close(lse, r["lse"], r["lse_tol"], "lse")
        for n, t in zip(("dq", "dk", "dv"), grads):
            ref.close(t, r[n], r[n + "_tol"], n)


@pytest.mark.parametrize("dtype", TYPES)
def test_hidden_nan_and_infinity(p3, cuda_device, dtype):
    """A NaN or an infinity in a row reaches exactly the results whose definition reads it.  The others are held to
    the definition without that row (a row that a product with 0 spoilt is computed again on another path, which
    rounds its probabilities elsewhere: both are within the tolerance of the definition, not of the same bits)."""
    dev = cuda_device
    lens, W, S = [90, 260], 40, 3
    for bad_row, value in ((200, float("nan")), (95, float("inf")), (349, float("nan"))):
        q, k, v, dout = inputs(lens, lens, 4, 2, dtype, dev, 7, pad=9)
        cfg = p3.make_seq_config(Hq=4, Hkv=2, window=W, sinks=S, dtype="bf16" if dtype == torch.bfloat16 else "f32")
        cu = offsets(lens, dev)
        r = ref.window(q[:350], k[:350], v[:350], lens, lens, W, S, cfg.softmax_scale, dout[:350])
        v[bad_row], k[bad_row] = value, value
        v[350:], k[350:], q[350:], dout[350:] = (float("nan"),) * 4      # rows of no sequence
        out, lse = p3.window_attn(cfg, q, k, v, cu)
        pos = torch.cat([torch.arange(n) for n in lens]).to(dev)
        seq = torch.tensor([0] * 90 + [1] * 260, device=dev)
        j, b = int(pos[bad_row]), int(seq[bad_row])
        reads = (seq == b) & (pos >= j) & ((pos - j < W) | (j < S))
        assert torch.isnan(out[:350][reads].float()).all()
        ref.close(out[:350][~reads], r["out"][~reads], r["out_tol"][~reads], "out")
        ref.close(lse[:350][~reads], r["lse"][~reads], r["lse_tol"][~reads], "lse")
        assert (out[350:] == 0).all()
        grads = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
        dq = grads[0][:350]
        assert torch.isnan(dq[reads].float()).any(-1).all()
        ref.close(dq[~reads], r["dq"][~reads], r["dq_tol"][~reads], "dq")
        # a key that only unspoilt queries see keeps its gradients
        spoilt = torch.zeros(350, dtype=torch.bool, device=dev)
        for i in torch.nonzero(reads).flatten().tolist():
            p = int(pos[i])
            spoilt |= (seq == b) & (pos <= p) & ((p - pos < W) | (pos < S))
        for g, n in zip(grads[1:], ("dk", "dv")):
            assert torch.isnan(g[:350][spoilt].float()).any(-1).all()
            ref.close(g[:350][~spoilt], r[n][~spoilt], r[n + "_tol"][~spoilt], n)
            assert (g[350:] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_hidden_query_nan(p3, cuda_device, dtype):
    """A NaN in one query's row (or its gradient's) spoils that row and the keys it sees, nothing else."""
    dev = cuda_device
    lens, W, S = [310], 32, 2
    for which in ("q", "dout"):
        q, k, v, dout = inputs(lens, lens, 4, 2, dtype, dev, 9)
        cfg = p3.make_seq_config(Hq=4, Hkv=2, window=W, sinks=S, dtype="bf16" if dtype == torch.bfloat16 else "f32")
        cu = offsets(lens, dev)
        r = ref.window(q, k, v, lens, lens, W, S, cfg.softmax_scale, dout)
        (q if which == "q" else dout)[150] = float("nan")
        out, lse = p3.window_attn(cfg, q, k, v, cu)
        grads = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
        rows = torch.arange(310, device=dev) == 150
        j = torch.arange(310, device=dev)
        keys = (j <= 150) & ((150 - j < W) | (j < S))
        assert torch.isnan(grads[0][rows].float()).all()
        ref.close(grads[0][~rows], r["dq"][~rows], r["dq_tol"][~rows], "dq")
        for g, n in zip(grads[1:], ("dk", "dv")):
            ref.close(g[~keys], r[n][~keys], r[n + "_tol"][~keys], n)
            assert torch.isnan(g[keys].float()).any(-1).all()


def test_rows_of_no_sequence(p3, cuda_device):
    """Rows before the first and behind the last sequence: kept in given outputs, 0 in new ones."""
    dev = cuda_device
    for dtype in TYPES:
        q, k, v, dout = inputs([150], [150], 8, 2, dtype, dev, 2)
        cfg = p3.make_seq_config(window=20, sinks=1, dtype="bf16" if dtype == torch.bfloat16 else "f32")
        cu = torch.tensor([10, 70, 121], dtype=torch.int32, device=dev)
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=dev)
        p3.window_attn(cfg, q, k, v, cu, out=out, lse=lse)
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout, *grads)
        new, new_lse = p3.window_attn(cfg, q, k, v, cu)
        new_grads = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
        for a, b, zero in [(out, new, 0.0), (lse, new_lse, -float("inf"))] + [(x, y, 0.0) for x, y in
                                                                            zip(grads, new_grads)]:
            assert torch.equal(a[10:121], b[10:121])
            for edge in (slice(0, 10), slice(121, None)):
                assert (a[edge] == 7.0).all() and (b[edge] == zero).all()
        r = ref.window(q[10:121], k[10:121], v[10:121], [60, 51], [60, 51], 20, 1, cfg.softmax_scale)
        ref.close(out[10:121], r["out"], r["out_tol"], "out")


def test_wrong_offsets_are_reported(p3, cuda_device):
    """Offsets out of order or out of range set the error bit; nothing outside the sequences' rows is written."""
    dev = cuda_device
    q, k, v, dout = inputs([64], [64], 8, 2, torch.bfloat16, dev)
    cfg = p3.make_seq_config(window=8)
    good = torch.tensor([0, 30, 64], dtype=torch.int32, device=dev)
    for cu in ([0, 40, 30], [0, 30, 65], [-1, 30, 64], [0, 2 ** 31 - 1, 64]):
        bad = torch.tensor(cu, dtype=torch.int32, device=dev)
        for cu_q, cu_k in ((bad, good), (good, bad), (bad, bad)):
            err = torch.zeros(1, dtype=torch.int32, device=dev)
            out, lse = p3.window_attn(cfg, q, k, v, cu_q, cu_k, err=err)
            assert int(err) == p3.DEVERR_LENGTHS and p3.check_status(err) == 9
            p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
            assert p3.check_status(err) == 9 and p3.check_status(err) == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_wrong_offsets_among_many_are_reported(p3, cuda_device, dtype):
    """Wherever the wrong offset of a large batch stands, some CTA sees it."""
    dev, B = cuda_device, 200
    q, k, v, dout = inputs([4 * B], [4 * B], 2, 1, dtype, dev)
    cfg = p3.make_seq_config(Hq=2, Hkv=1, window=8, sinks=2, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    good = torch.arange(B + 1, dtype=torch.int32, device=dev) * 4
    for at in (0, 1, 31, 32, 33, 100, 199, 200):
        for value in (-5, 4 * B + 1, 2 ** 31 - 1):
            bad = good.clone()
            bad[at] = value
            for cu_q, cu_k in ((bad, good), (good, bad)):
                err = torch.zeros(1, dtype=torch.int32, device=dev)
                out, lse = p3.window_attn(cfg, q, k, v, cu_q, cu_k, err=err)
                assert p3.check_status(err) == 9
                p3.window_attn_bwd(cfg, q, k, v, cu_q, cu_k, out, lse, dout, err=err)
                assert p3.check_status(err) == 9


def test_rows_of_no_sequence_of_many(p3, cuda_device):
    """The rows outside, many before and behind a batch of many sequences."""
    dev, B = cuda_device, 100
    for dtype in TYPES:
        q, k, v, dout = inputs([3000], [3000], 2, 1, dtype, dev, 2)
        cfg = p3.make_seq_config(Hq=2, Hkv=1, window=20, dtype="bf16" if dtype == torch.bfloat16 else "f32")
        cu = torch.arange(B + 1, dtype=torch.int32, device=dev) * 7 + 900
        out, lse = p3.window_attn(cfg, q, k, v, cu)
        grads = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
        for t, zero in ((out, 0.0), (lse, -float("inf"))) + tuple((g, 0.0) for g in grads):
            assert (t[:900] == zero).all() and (t[1600:] == zero).all() and (t[900:1600] != zero).any()


def test_autograd_and_same_bits(p3, cuda_device):
    """window_attention's gradients are window_attn_bwd's, twice the same bits, with a strided output gradient too."""
    dev = cuda_device
    lens = [333, 90]
    q, k, v, dout = inputs(lens, lens, 8, 2, torch.bfloat16, dev, 4)
    cfg = p3.make_seq_config(window=64, sinks=4)
    cu = offsets(lens, dev)
    out, lse = p3.window_attn(cfg, q, k, v, cu)
    want = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
    for strided in (False, True):
        leaves = [t.detach().requires_grad_(True) for t in (q, k, v)]
        o = p3.window_attention(cfg, *leaves, cu)
        assert torch.equal(o, out)
        d = dout.transpose(0, 1).contiguous().transpose(0, 1) if strided else dout
        got = torch.autograd.grad(o, leaves, d)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_difference_quotient(p3, cuda_device):
    """The float gradients against central differences of the float forward, along a random direction.  The loss is
    a sum of n = 60 * 4 * 64 products of values of order 1, computed in 64 bits from outputs that are off by at most
    r["out_tol"]; the quotient divides that by the step."""
    dev = cuda_device
    q, k, v, dout = inputs([60], [60], 4, 2, torch.float32, dev, 6)
    cfg = p3.make_seq_config(Hq=4, Hkv=2, window=17, sinks=1, dtype="f32")
    cu = offsets([60], dev)
    out, lse = p3.window_attn(cfg, q, k, v, cu)
    grads = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
    r = ref.window(q, k, v, [60], [60], 17, 1, cfg.softmax_scale, dout)
    step = 2.0 ** -6
    for i, (name, t) in enumerate(zip(("dq", "dk", "dv"), (q, k, v))):
        d = torch.randn(t.shape, device=dev, generator=torch.Generator(device=dev).manual_seed(i))
        d = torch.round(d * 16) / 16          # t + step * d is a float again, up to its own last bits
        ends = []
        for s in (step, -step):
            args = [q, k, v]
            args[i] = t + s * d
            ends.append(float((p3.window_attn(cfg, *args, cu)[0].double() * dout.double()).sum()))
            exact = ref.window(*args, [60], [60], 17, 1, cfg.softmax_scale)["out"]
            assert abs(ends[-1] - float((exact * dout.double()).sum())) <= float((r["out_tol"] * 4 * dout.abs()).sum())
        got = float((grads[i].double() * d.double()).sum())
        # the third derivative's term, from the quotient at half the step in 64 bits
        halves = []
        for s in (step / 2, -step / 2):
            args = [q.double(), k.double(), v.double()]
            args[i] = args[i] + s * d.double()
            o = ref.window(*[a.float() for a in args], [60], [60], 17, 1, cfg.softmax_scale)["out"]
            halves.append(float((o * dout.double()).sum()))
        quotient, half = (ends[0] - ends[1]) / (2 * step), (halves[0] - halves[1]) / step
        noise = float((r["out_tol"] * 4 * dout.abs()).sum()) / step
        assert abs(got - quotient) <= 2 * abs(quotient - half) + 2 * noise + float((r[name + "_tol"] * d.abs()).sum())


# ---- the cache ------------------------------------------------------------------------

def make_cache(lengths, page, Hkv, dtype, dev, seed=0, spare=0, extra=1):
    """Pools of NaN with normal rows in the used slots, pages in random order; the table's unused entries are -1."""
    g = torch.Generator(device=dev).manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare + 2
    wide = max(need + [1]) + extra
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lengths), wide), -1, dtype=torch.int32)
    k = torch.full((pages, page, Hkv, 64), float("nan"), dtype=dtype, device=dev)
    v = k.clone()
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        for t in (k, v):
            rows = t[order[at:at + n].to(dev)].view(-1, Hkv, 64)
            rows[:lengths[b]] = torch.randn(lengths[b], Hkv, 64, generator=g, device=dev).to(dtype)
            t[order[at:at + n].to(dev)] = rows.view(-1, page, Hkv, 64)
        at += n
    return k, v, table.to(dev), torch.tensor(lengths, dtype=torch.int32, device=dev), order[at:]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,page,Hq,Hkv,W,S", [
    ([1], 16, 8, 2, 0, 0), ([0], 16, 8, 2, 0, 0), ([0, 5, 0, 16, 17], 16, 4, 1, 0, 0),
    ([63, 64, 65, 1], 64, 8, 1, 0, 0), ([1000, 3, 257], 32, 8, 8, 0, 0), ([5000], 64, 8, 2, 0, 0),
    ([900, 40], 16, 4, 4, 100, 3), ([777, 100, 101, 99], 256, 2, 1, 100, 0), ([300], 128, 6, 3, 1, 64),
    ([4097, 1, 2048] + [7] * 40, 64, 16, 2, 0, 0), ([20000, 11], 64, 1, 1, 0, 0), ([700] * 9, 32, 16, 4, 333, 17),
])
def test_decode(p3, cuda_device, lengths, page, Hq, Hkv, W, S, dtype):
    """Unused slots hold NaN and unused table entries -1: neither is read.  With and without the weights."""
    dev = cuda_device
    k, v, table, n, _ = make_cache(lengths, page, Hkv, dtype, dev)
    q = torch.randn(len(lengths), Hq, 64, device=dev, generator=torch.Generator(device=dev).manual_seed(1)).to(dtype)
    cfg = p3.make_seq_config(Hq=Hq, Hkv=Hkv, window=W, sinks=S, page=page,
                             dtype="bf16" if dtype == torch.bfloat16 else "f32")
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = p3.cache_attn(cfg, q, k, v, table, n, err=err)
    weights = torch.full((len(lengths), table.shape[1] * page), 3.0, device=dev)
    out2, lse2 = p3.cache_attn(cfg, q, k, v, table, n, weights=weights, err=err)
    added = torch.full_like(weights, 2.0)
    p3.cache_attn(cfg, q, k, v, table, n, weights=added, accumulate=True, err=err)
    assert p3.check_status(err) == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    r = ref.decode(q, k, v, table, n, W, S, cfg.softmax_scale)
    ref.close(out, r["out"], r["out_tol"], "out")
    ref.close(lse, r["lse"], r["lse_tol"], "lse")
    inside = torch.arange(weights.shape[1], device=dev)[None] < n[:, None]
    ref.close(weights[inside], r["weights"][inside], r["weights_tol"][inside], "weights")
    assert (weights[~inside] == 3.0).all() and (added[~inside] == 2.0).all()
    # one addition in 32 bits to 2
    ref.close(added[inside], r["weights"][inside] + 2.0, r["weights_tol"][inside] + 2.0 ** -24 * (2 + Hq), "added")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,page", [([50, 9], 16), ([3000, 700, 1], 64)], ids=["short", "split"])
def test_decode_where_no_score_is_finite(p3, cuda_device, lengths, page, dtype):
    """Heads whose visible scores are all -infinity: output 0, log-sum-exp -infinity and no weight; the other heads and
    sequences as ever.  With accumulate nothing but their weights is added."""
    dev = cuda_device
    k, v, table, n, _ = make_cache(lengths, page, 2, dtype, dev)
    q = torch.randn(len(lengths), 8, 64, device=dev, generator=torch.Generator(device=dev).manual_seed(1)).to(dtype)
    cfg = p3.make_seq_config(page=page, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    r = ref.decode(q[:, 4:], k[:, :, 1:], v[:, :, 1:], table, n, 0, 0, cfg.softmax_scale)
    # key head 0: -infinity in one dim of every row of the first sequence, met by a positive query there
    used = table[0, :-(-lengths[0] // page)].long()
    k[used, :, 0, 7] = -float("inf")
    q[:, :4, 7] = 1.0
    whole = ref.decode(q[1:], k, v, table[1:], n[1:], 0, 0, cfg.softmax_scale)
    weights = torch.zeros(len(lengths), table.shape[1] * page, device=dev)
    out, lse = p3.cache_attn(cfg, q, k, v, table, n, weights=weights)
    added = torch.full_like(weights, 2.0)
    p3.cache_attn(cfg, q, k, v, table, n, weights=added, accumulate=True)
    assert (out[0, :4] == 0).all() and (lse[0, :4] == -float("inf")).all()
    ref.close(out[:, 4:], r["out"], r["out_tol"], "out")
    ref.close(out[1:], whole["out"], whole["out_tol"], "out")
    ref.close(weights[0], r["weights"][0], r["weights_tol"][0], "weights")
    ref.close(weights[1:], whole["weights"], whole["weights_tol"], "weights")
    inside = torch.arange(weights.shape[1], device=dev)[None] < n[:, None]
    assert (added[~inside] == 2.0).all()
    ref.close(added[0], r["weights"][0] + 2.0, r["weights_tol"][0] + 2.0 ** -24 * 10, "added")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,longest", [(512, 3000), (511, 3000), (511, 1000)])
def test_decode_at_the_splits_borders(p3, cuda_device, batch, longest, dtype):
    """4,096 (sequence, key head) pairs and fewer, capacities of 1,024 slots and more: one long sequence among short
    ones, split over the GPU or not."""
    dev = cuda_device
    lengths = [(7 * i) % 20 for i in range(batch)]
    lengths[batch // 3] = longest
    k, v, table, n, _ = make_cache(lengths, 16, 8, dtype, dev)
    q = torch.randn(batch, 8, 64, device=dev, generator=torch.Generator(device=dev).manual_seed(1)).to(dtype)
    cfg = p3.make_seq_config(Hq=8, Hkv=8, page=16, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = p3.cache_attn(cfg, q, k, v, table, n, err=err)
    assert p3.check_status(err) == 0
    some = sorted(set(range(0, batch, 9)) | {batch // 3 + d for d in (-1, 0, 1)} | {batch - 1})
    r = ref.decode(q[some], k, v, table[some], n[some], 0, 0, cfg.softmax_scale)
    ref.close(out[some], r["out"], r["out_tol"], "out")
    ref.close(lse[some], r["lse"], r["lse_tol"], "lse")


def test_decode_is_window_attention_of_one_query(p3, cuda_device):
    """The same tokens through the packed operator and through the cache."""
    dev = cuda_device
    lens, W, S = [800, 31, 64], 200, 4
    cfg = p3.make_seq_config(window=W, sinks=S, page=32)
    q, k, v, _ = inputs([1] * 3, lens, 8, 2, torch.bfloat16, dev, 3)
    out, lse = p3.window_attn(cfg, q, k, v, offsets([1] * 3, dev), offsets(lens, dev))
    cache = p3.PagedCache(cfg, 3, 832)
    cache.append(k, v, offsets(lens, dev))
    got, got_lse = p3.cache_attn(cfg, q, cache.k_pages, cache.v_pages, cache.table, cache.lengths)
    cache.check()
    r = ref.window(q, k, v, [1] * 3, lens, W, S, cfg.softmax_scale)
    for o, l in ((out, lse), (got, got_lse)):
        ref.close(o, r["out"], r["out_tol"], "out")
        ref.close(l, r["lse"], r["lse_tol"], "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,Hq,Hkv", [([300, 7], 8, 2), ([5000, 0, 90], 8, 2), ([3] * 300 + [2000], 4, 2)])
def test_results_next_to_and_over_the_queries(p3, cuda_device, lengths, Hq, Hkv, dtype):
    """Outputs that lie right behind the inputs in one buffer, and attention over the cache whose output takes its
    queries' place: the same bits."""
    dev, B = cuda_device, len(lengths)
    k, v, table, n, _ = make_cache(lengths, 64, Hkv, dtype, dev)
    q = torch.randn(B, Hq, 64, device=dev, generator=torch.Generator(device=dev).manual_seed(1)).to(dtype)
    cfg = p3.make_seq_config(Hq=Hq, Hkv=Hkv, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    want, lse = p3.cache_attn(cfg, q, k, v, table, n)
    both = torch.empty(2, B, Hq, 64, dtype=dtype, device=dev)
    both[0] = q
    got, got_lse = p3.cache_attn(cfg, both[0], k, v, table, n, out=both[1])
    assert torch.equal(got, want) and torch.equal(got_lse, lse) and torch.equal(both[0], q)
    got, got_lse = p3.cache_attn(cfg, both[0], k, v, table, n, out=both[0])
    assert got is not want and torch.equal(got, want) and torch.equal(got_lse, lse)
    with pytest.raises(p3.Pack3DError, match="INVALID_ARG"):
        p3.cache_attn(cfg, both.view(-1, Hq, 64)[:B], k, v, table, n, out=both.view(-1, Hq, 64)[1:B + 1])
    with pytest.raises(p3.Pack3DError, match="INVALID_ARG"):
        w = torch.rand(B, table.shape[1] * 64, device=dev)
        p3.cache_evict(cfg, k, v, table, n, w, table, 64, 0, new_weights=w, new_lengths=torch.empty_like(n),
                       kept=torch.empty(B, 64, dtype=torch.int32, device=dev))


def test_an_empty_buffer_lies_over_nothing(p3, cuda_device):
    """No query rows: their buffers hold nothing, wherever the pointers point."""
    import ctypes
    dev = cuda_device
    k, v, dk, dv = (torch.full((40, 2, 64), 3.0, dtype=torch.bfloat16, device=dev) for _ in range(4))
    cu_q, cu_k = offsets([0], dev), offsets([40], dev)
    cfg = p3.make_seq_config()
    ws = torch.empty(max(256, p3.window_attn_bwd_workspace_bytes(cfg, 1, 0, 40)), dtype=torch.uint8, device=dev)
    inside = dk.data_ptr() + 64
    st = p3.lib.pack3d_window_attn_bwd(ctypes.byref(cfg), 1, 0, 40, cu_q.data_ptr(), cu_k.data_ptr(), inside, k.data_ptr(),
                                       v.data_ptr(), inside, inside, inside, inside, dk.data_ptr(), dv.data_ptr(), 0,
                                       ws.data_ptr(), ws.numel(), None, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and (dk == 0).all() and (dv == 0).all()


def test_pool_beyond_32_bit_offsets(p3, cuda_device):
    """Pages whose elements and bytes lie beyond 2^31 and 2^32: written, read and moved there.  (Keys and values in
    one pool of 10.5 GB: append writes equal rows to both.)"""
    dev = cuda_device
    page, Hkv, pages, n = 256, 8, 40000, 700
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("less than 16 GB free")
    pool = torch.empty(pages, page, Hkv, 64, dtype=torch.bfloat16, device=dev)
    table = torch.tensor([[39999, 33000, 17]], dtype=torch.int32, device=dev)
    new_table = torch.tensor([[39001, 39000]], dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(5)
    k = torch.randn(n, Hkv, 64, generator=g, device=dev).bfloat16()
    q = torch.randn(1, Hkv, 64, generator=g, device=dev).bfloat16()
    cfg = p3.make_seq_config(Hq=Hkv, Hkv=Hkv, page=page)
    zero, used = (torch.tensor([x], dtype=torch.int32, device=dev) for x in (0, n))
    p3.cache_append(cfg, k, k, pool, pool, table, zero, offsets([n], dev))
    assert torch.equal(pool[table[0].long()].view(-1, Hkv, 64)[:n], k)
    weights = torch.zeros(1, 3 * page, device=dev)
    out, lse = p3.cache_attn(cfg, q, pool, pool, table, used, weights=weights)
    r = ref.window(q, k, k, [1], [n], 0, 0, cfg.softmax_scale)
    ref.close(out, r["out"], r["out_tol"], "out")
    ref.close(lse, r["lse"], r["lse_tol"], "lse")
    kept, _, lengths = p3.cache_evict(cfg, pool, pool, table, used, weights, new_table, 300, 10)
    want = ref.evict(used, weights.cpu(), 300, 0, 10)[0]
    assert kept[0].tolist() == want and int(lengths) == 300
    assert torch.equal(pool[new_table[0].long()].view(-1, Hkv, 64)[:300], k[torch.tensor(want, device=dev)])


def test_decode_reports_bad_pages_and_lengths(p3, cuda_device):
    """A page outside the pool or a length outside the capacity: reported, and no address outside the pool is read
    (the kernel checks every page number before it is used)."""
    dev = cuda_device
    for dtype in TYPES:
        k, v, table, n, _ = make_cache([100, 50], 16, 2, dtype, dev)
        q = torch.zeros(2, 8, 64, device=dev, dtype=dtype)
        cfg = p3.make_seq_config(page=16, dtype="bf16" if dtype == torch.bfloat16 else "f32")
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        for page in (-1, k.shape[0], 2 ** 31 - 1):
            t = table.clone()
            t[1, 2] = page
            w = torch.zeros(2, t.shape[1] * 16, device=dev)
            p3.cache_attn(cfg, q, k, v, t, n, weights=w, err=err)
            assert p3.check_status(err) == 10
        for length in (-1, table.shape[1] * 16 + 1):
            m = n.clone()
            m[0] = length
            full = torch.zeros_like(table)     # every page of the table is in the pool
            p3.cache_attn(cfg, q, k, v, full, m, err=err)
            assert p3.check_status(err) == 9


@pytest.mark.parametrize("dtype", TYPES)
def test_append(p3, cuda_device, dtype):
    dev = cuda_device
    for lengths, new, page, Hkv in (([0, 15, 16, 17], None, 16, 2), ([3, 0, 100, 64], [40, 0, 1, 130], 64, 1),
                                    ([5], [300], 32, 3)):
        rows = len(lengths) if new is None else sum(new)
        total = [a + b for a, b in zip(lengths, new or [1] * len(lengths))]
        k, v, table, _, _ = make_cache(total, page, Hkv, dtype, dev, extra=0)
        n = torch.tensor(lengths, dtype=torch.int32, device=dev)
        a, b = (torch.randn(rows + 5, Hkv, 64, device=dev).to(dtype) for _ in range(2))
        cu = None if new is None else offsets(new, dev)
        if cu is None:
            a, b = a[:rows].contiguous(), b[:rows].contiguous()      # otherwise the last five rows are no sequence's
        cfg = p3.make_seq_config(Hq=Hkv, Hkv=Hkv, page=page, dtype="bf16" if dtype == torch.bfloat16 else "f32")
        want_k, want_v = k.clone(), v.clone()
        at = 0
        for s, (old, m) in enumerate(zip(lengths, new or [1] * len(lengths))):
            for i in range(m):
                p = int(table[s, (old + i) // page])
                want_k[p, (old + i) % page], want_v[p, (old + i) % page] = a[at], b[at]
                at += 1
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        p3.cache_append(cfg, a, b, k, v, table, n, cu, err=err)
        assert p3.check_status(err) == 0
        for got, want in ((k, want_k), (v, want_v)):
            assert torch.equal(torch.nan_to_num(got, nan=9.0), torch.nan_to_num(want, nan=9.0))


def test_append_reports_offsets_that_no_row_meets(p3, cuda_device):
    dev = cuda_device
    cfg = p3.make_seq_config(Hq=2, Hkv=1, page=16)
    pages = [torch.zeros(12, 16, 1, 64, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    table = torch.arange(12, dtype=torch.int32, device=dev).view(3, 4)
    lengths = torch.zeros(3, dtype=torch.int32, device=dev)
    rows = torch.randn(20, 1, 64, device=dev).bfloat16()
    for cu, want in (([0, 10, 5, 20], p3.DEVERR_LENGTHS), ([0, 10, 15, 21], p3.DEVERR_LENGTHS), ([0, 10, 10, 20], 0)):
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        p3.cache_append(cfg, rows, rows, *pages, table, lengths, torch.tensor(cu, dtype=torch.int32, device=dev),
                        err=err)
        assert int(err) == want


def test_append_reports_what_does_not_fit(p3, cuda_device):
    """Rows behind the capacity, negative lengths, pages outside the pool and wrong offsets: reported, not written."""
    dev = cuda_device
    cfg = p3.make_seq_config(page=16)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    rows = torch.ones(2, 2, 64, device=dev, dtype=torch.bfloat16)

    def call(table, lengths, cu=None):
        k = torch.zeros(4, 16, 2, 64, device=dev, dtype=torch.bfloat16)
        v = torch.zeros_like(k)
        p3.cache_append(cfg, rows, rows, k, v, torch.tensor(table, dtype=torch.int32, device=dev),
                        torch.tensor(lengths, dtype=torch.int32, device=dev),
                        None if cu is None else torch.tensor(cu, dtype=torch.int32, device=dev), err=err)
        return p3.check_status(err), int((k.float().sum(-1) != 0).sum()) // 2, int((v.float().sum(-1) != 0).sum()) // 2

    assert call([[0, 1], [2, 3]], [31, 32]) == (9, 1, 1)
    assert call([[0, 1], [2, 3]], [-1, 0]) == (9, 1, 1)
    assert call([[0, 4], [-1, 3]], [16, 0]) == (10, 0, 0)
    assert call([[0, 1], [2, 3]], [0, 0], [0, 3, 2])[0] == 9
    assert call([[0, 1], [2, 3]], [0, 0], [0, 1, 2]) == (0, 2, 2)
    assert call([[0, 1], [2, 3]], [2 ** 31 - 1, 0], [0, 2, 2]) == (9, 0, 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,page,budget,sinks,recent,kind", [
    ([100, 40, 0, 64, 65], 16, 64, 4, 10, "random"), ([3000], 64, 1000, 0, 0, "random"),
    ([3000, 2999], 32, 1024, 64, 900, "ties"), ([500], 16, 70, 6, 64, "all equal"), ([500], 16, 1, 0, 0, "ties"),
    ([500, 200], 16, 80, 0, 80, "random"), ([20000, 70], 64, 8192, 4, 128, "ties"), ([90], 16, 50, 0, 5, "odd values"),
])
def test_evict(p3, cuda_device, lengths, page, budget, sinks, recent, kind, dtype):
    dev = cuda_device
    new_wide = -(-budget // page) + 1
    k, v, table, n, spare = make_cache(lengths, page, 2, dtype, dev, spare=new_wide * len(lengths))
    new_table = spare[:new_wide * len(lengths)].view(len(lengths), new_wide).int().to(dev)
    cap = table.shape[1] * page
    g = torch.Generator(device=dev).manual_seed(3)
    w = torch.exp(2 * torch.randn(len(lengths), cap, generator=g, device=dev))
    if kind == "ties":
        w = torch.floor(w * 4) / 4
    elif kind == "all equal":
        w = torch.full_like(w, 0.25)
    elif kind == "odd values":
        odd = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-40, -1.0, 3.0], device=dev)
        w = odd[torch.randint(0, 8, w.shape, generator=g, device=dev)]
    cfg = p3.make_seq_config(Hq=2, Hkv=2, sinks=sinks, page=page, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    before_k, before_v = k.clone(), v.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kept, nw, nl = p3.cache_evict(cfg, k, v, table, n, w, new_table, budget, recent, err=err)
    assert p3.check_status(err) == 0
    want = ref.evict(n, w.cpu(), budget, sinks, recent)
    written = torch.zeros(k.shape[0], page, dtype=torch.bool, device=dev)
    for b, rows in enumerate(want):
        assert int(nl[b]) == len(rows)
        assert kept[b].tolist() == rows + [-1] * (budget - len(rows))
        idx = torch.tensor(rows, dtype=torch.long, device=dev)
        assert torch.equal(torch.nan_to_num(nw[b, :len(rows)], nan=9.0), torch.nan_to_num(w[b, idx], nan=9.0))
        assert (nw[b, len(rows):] == 0).all()
        at = torch.arange(len(rows), device=dev)
        dst, src = new_table[b, at // page].long(), table[b, idx // page].long()
        for after, before in ((k, before_k), (v, before_v)):
            assert torch.equal(after[dst, at % page], before[src, idx % page])
        written[dst, at % page] = True
    for after, before in ((k, before_k), (v, before_v)):
        assert torch.equal(torch.nan_to_num(after[~written], nan=9.0), torch.nan_to_num(before[~written], nan=9.0))


def test_evict_reports_bad_pages(p3, cuda_device):
    dev = cuda_device
    cfg = p3.make_seq_config(Hq=2, Hkv=2, page=16)
    k, v, table, n, spare = make_cache([100], 16, 2, torch.bfloat16, dev, spare=4)
    new = spare[:4].view(1, 4).int().to(dev)
    w = torch.rand(1, table.shape[1] * 16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    for which in ("old", "new"):
        t, u = table.clone(), new.clone()
        (t if which == "old" else u)[0, 3] = k.shape[0]       # slots 48 .. 63: among the recent ones
        p3.cache_evict(cfg, k, v, t, n, w, u, 64, 60, err=err)
        assert p3.check_status(err) == 10
    p3.cache_evict(cfg, k, v, table, n + 10000, w, new, 64, 0, err=err)
    assert p3.check_status(err) == 9


# ---- together, as they are used ------------------------------------------------------------

def test_prompts_tokens_and_eviction_together(p3, cuda_device):
    """Prompts through the packed operator and into the cache, several tokens one at a time, an eviction by the
    collected weights, and more tokens: every output against the definition over the tokens that are left."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(12)
    lens, budget, recent = [150, 31, 90], 64, 16
    cfg = p3.make_seq_config(Hq=4, Hkv=2, sinks=2, page=16, dtype="f32")
    cache = p3.PagedCache(cfg, 3, 256, budget=budget)

    def rows(n, heads):
        return torch.randn(n, heads, 64, generator=g, device=dev)

    q, k, v = rows(sum(lens), 4), rows(sum(lens), 2), rows(sum(lens), 2)
    cu = offsets(lens, dev)
    out, lse = p3.window_attn(cfg, q, k, v, cu)
    r = ref.window(q, k, v, lens, lens, 0, 2, cfg.softmax_scale)
    ref.close(out, r["out"], r["out_tol"], "prompt")
    cache.append(k, v, cu)
    keys = [list(x.split(1)) for x in k.split(lens)]
    values = [list(x.split(1)) for x in v.split(lens)]
    total = [torch.zeros(n, dtype=torch.float64, device=dev) for n in lens]

    def step():
        k1, v1, q1 = rows(3, 2), rows(3, 2), rows(3, 4)
        cache.append(k1, v1)
        got = cache.attend(q1)
        for b in range(3):
            keys[b].append(k1[b:b + 1])
            values[b].append(v1[b:b + 1])
        klens = [len(x) for x in keys]
        r = ref.window(q1, torch.cat([x for y in keys for x in y]), torch.cat([x for y in values for x in y]), [1] * 3,
                       klens, 0, 2, cfg.softmax_scale)
        ref.close(got, r["out"], r["out_tol"], "token")
        for b in range(3):
            K = torch.cat(keys[b]).double()
            p = sum(torch.softmax(K[:, h // 2] @ q1[b, h].double() * cfg.softmax_scale, 0) for h in range(4))
            total[b] = torch.cat([total[b], torch.zeros(1, dtype=torch.float64, device=dev)]) + p

    for _ in range(5):
        step()
    for b in range(3):
        n = len(keys[b])
        # five sums of four probabilities in 32 bits, each off by far less than 2^-24 times its terms' number
        assert (cache.weights[b, :n].double() - total[b]).abs().max() <= 2.0 ** -24 * 20 * (200 + 66 * 16)
    want = ref.evict(cache.lengths, cache.weights.cpu(), budget, 2, recent)
    kept = cache.evict(recent)
    for b in range(3):
        assert kept[b].tolist() == want[b] + [-1] * (budget - len(want[b]))
        keys[b], values[b] = [keys[b][j] for j in want[b]], [values[b][j] for j in want[b]]
        total[b] = total[b][torch.tensor(want[b], device=dev)]
        assert int(cache.lengths[b]) == len(want[b])
    for _ in range(20):      # past the next page's end
        step()
    cache.evict(recent)
    step_lengths = cache.lengths.tolist()
    assert step_lengths == [64, 56, 64]
    cache.check()
