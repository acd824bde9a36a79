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
