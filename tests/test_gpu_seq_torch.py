"""The sequence operators inside PyTorch: saved-tensor hooks, fake tensors."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def p3(cuda_device):
    import geometry_aware_local_b200 as p3
    return p3


def tensors(n, Hq, Hkv, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(n, h, 64, generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv, Hq)]


def transposed(t):
    """Equal values, other strides."""
    return t.transpose(0, 1).contiguous().transpose(0, 1) if t.dim() > 1 else t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_saved_tensors_of_another_layout(p3, dtype):
    """What a hook gives back in place of a saved tensor may have other strides: the gradients stay right."""
    q, k, v, dout = tensors(300, 8, 2, dtype)
    cfg = p3.make_seq_config(window=64, sinks=4, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    cu = torch.tensor([0, 180, 300], dtype=torch.int32, device="cuda")
    out, lse = p3.window_attn(cfg, q, k, v, cu)
    want = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
    for pack, unpack in ((lambda t: t, transposed), (transposed, lambda t: t),
                         (lambda t: t.cpu(), lambda t: t.to("cuda"))):
        leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
        with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
            o = p3.window_attention(cfg, *leaves, cu)
        for a, b in zip(torch.autograd.grad(o, leaves, dout), want):
            assert a.is_contiguous() and torch.equal(a, b)


@pytest.mark.parametrize("unpack,match", [
    (lambda t: t.half() if t.dim() == 3 else t, "must be"),          # half as many bytes in float
    (lambda t: t.cpu(), "CUDA"), (lambda t: t[:-1] if t.dim() > 1 else t, "shape"),
    (lambda t: t.long() if t.dtype == torch.int32 else t, "must be"),
], ids=["type", "device", "rows", "offsets"])
def test_saved_tensors_that_are_something_else(p3, unpack, match):
    q, k, v, dout = tensors(64, 8, 2, torch.float32)
    cfg = p3.make_seq_config(window=16, dtype="f32")
    cu = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    leaves = [t.requires_grad_(True) for t in (q, k, v)]
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        o = p3.window_attention(cfg, *leaves, cu)
    with pytest.raises(ValueError, match=match):
        torch.autograd.grad(o, leaves, dout)


def test_a_call_with_fake_tensors_leaves_nothing_behind(p3, monkeypatch):
    """Under FakeTensorMode there is no memory to run on: the call is refused, and the next one, on tensors that exist,
    makes its results and workspaces of memory that exists too."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    monkeypatch.setattr(p3.seq, "_templates", {})        # as in a new process
    q, k, v, dout = tensors(100, 8, 2)
    cfg = p3.make_seq_config(window=16, sinks=2, page=16)
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    with FakeTensorMode() as mode, pytest.warns(UserWarning, match="data pointer"):
        with pytest.raises(p3.Pack3DError):
            p3.window_attn(cfg, *(mode.from_tensor(t) for t in (q, k, v, cu)))
    out, lse = p3.window_attn(cfg, q, k, v, cu)
    grads = p3.window_attn_bwd(cfg, q, k, v, cu, None, out, lse, dout)
    cache = p3.PagedCache(cfg, 1, 2048, budget=32)
    cache.append(k, v, cu)
    got, got_lse = p3.cache_attn(cfg, q[99:], cache.k_pages, cache.v_pages, cache.table, cache.lengths)
    kept = cache.evict(8)
    cache.check()
    for t in (out, lse, *grads, got, got_lse, kept):
        assert type(t) is torch.Tensor and t.data_ptr() != 0
    ref_lse = torch.logsumexp((q[99].double().view(2, 4, 64) @ torch.cat((k[:2], k[84:])).double().permute(1, 2, 0)) / 8, -1)
    assert torch.allclose(lse[99].double(), ref_lse.view(-1), atol=1e-4)
    assert torch.allclose(got_lse[0].double(), ref_lse.view(-1), atol=1e-4)


def test_a_first_call_in_inference_mode(p3, monkeypatch):
    """What the first call of a process leaves behind does not make later results inference tensors."""
    monkeypatch.setattr(p3.seq, "_templates", {})
    q, k, v, dout = tensors(100, 8, 2)
    cfg, cu = p3.make_seq_config(window=16), torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    with torch.inference_mode():
        want, lse = p3.window_attn(cfg, q, k, v, cu)
        grads = p3.window_attn_bwd(cfg, q, k, v, cu, None, want, lse, dout)
    leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
    out = p3.window_attention(cfg, *leaves, cu)
    assert torch.equal(out, want)
    for a, b in zip(torch.autograd.grad(out, leaves, dout), grads):
        assert torch.equal(a, b) and not a.is_inference()
    assert not p3.window_attn(cfg, q, k, v, cu)[1].is_inference()
