"""Python binding of the causal sequence operators (``include/pack3d_seq.h``): windowed attention of packed
sequences with its gradients, and the paged key-value cache that serves the same attention one token at a time.

Typical use (tensors CUDA and contiguous, q [rows,Hq,64], k and v [rows,Hkv,64], cu int32 [batch+1])::

    import geometry_aware_local_b200 as p3
    cfg = p3.make_seq_config(window=1024, sinks=4)       # Hq=8, Hkv=2, bf16
    out = p3.window_attention(cfg, q, k, v, cu)          # differentiable in q, k and v
    out, lse = p3.window_attn(cfg, q, k, v, cu)          # without gradients

    cache = p3.PagedCache(cfg, batch=16, capacity=8192, budget=4096)
    cache.append(k, v, cu)                               # the prompts
    out = cache.attend(q1)                               # q1 [16,Hq,64], one new token each (appended before)
    cache.evict(recent=512)                              # by the attention weight collected by attend
    cache.check()

Every function runs asynchronously on the current stream of its tensors' device, whichever device is current.  With
an explicit ``stream`` the caller also gives every output and the workspace, since memory allocated here belongs to
the current stream.  ``err`` is an int32 error word on the device (zeroed by the caller before its first use), read
by ``check_status``; without one, errors that only the device can see (offsets, lengths or page numbers out of
range, a wait that ran out) go unreported, and the results are then whatever was in their memory.

Sums, softmax and its statistics are in float whatever the type; with bf16 the probabilities, and in the backward the
scores' gradients, are rounded to bf16 for the tensor cores' second product, as the results are at the end.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

from . import BF16, F32, Pack3DError, check_status, lib

ERR_WORKSPACE = 6     # PACK3D_ERR_WORKSPACE

DH = 64


class SeqConfig(ctypes.Structure):
    """Mirror of ``pack3d_seq_config``."""
    _fields_ = [("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d_h", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("page", ctypes.c_int32), ("flags", ctypes.c_int32), ("wait_limit_us", ctypes.c_int32),
                ("reserved0", ctypes.c_int32), ("reserved1", ctypes.c_int32)]


SEQ_ENTRY_POINTS = ("pack3d_default_seq_config", "pack3d_validate_seq_config", "pack3d_window_attn",
                    "pack3d_window_attn_bwd_workspace_bytes", "pack3d_window_attn_bwd", "pack3d_cache_append",
                    "pack3d_cache_attn_workspace_bytes", "pack3d_cache_attn", "pack3d_cache_evict")


def _sign():
    P, I32, I64, C, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(SeqConfig), ctypes.c_size_t
    sig = {
        "pack3d_default_seq_config": (None, [C]),
        "pack3d_validate_seq_config": (ctypes.c_int, [C]),
        "pack3d_window_attn": (ctypes.c_int, [C, I32, I64, I64] + [P] * 7 + [I32, P, P]),
        "pack3d_window_attn_bwd_workspace_bytes": (S, [C, I32, I64, I64]),
        "pack3d_window_attn_bwd": (ctypes.c_int, [C, I32, I64, I64] + [P] * 11 + [I32, P, S, P, P]),
        "pack3d_cache_append": (ctypes.c_int, [C, I32, I64, P, P, P, I32, I32] + [P] * 6),
        "pack3d_cache_attn_workspace_bytes": (S, [C, I32, I32, I32]),
        "pack3d_cache_attn": (ctypes.c_int, [C, I32, P, P, P, P, I32, I32, P, P, P, P, I32, P, S, P, P]),
        "pack3d_cache_evict": (ctypes.c_int, [C, I32, P, P, I32, P, I32, P, P, I32, I32, P, I32, P, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


_sign()


def make_seq_config(*, Hq: int = 8, Hkv: int = 2, d_h: int = DH, window: int = 0, sinks: int = 0, page: int = 64,
                    softmax_scale: Optional[float] = None, dtype: str = "bf16", flags: int = 0,
                    wait_limit_us: int = 0) -> SeqConfig:
    c = SeqConfig()
    c.Hq, c.Hkv, c.d_h = Hq, Hkv, d_h
    c.dtype = BF16 if dtype in ("bf16", BF16) else F32
    c.softmax_scale = 1.0 / math.sqrt(d_h) if softmax_scale is None else softmax_scale
    c.window, c.sinks, c.page = window, sinks, page
    c.flags, c.wait_limit_us = flags, wait_limit_us
    return c


def validate_seq(cfg: SeqConfig) -> int:
    return lib.pack3d_validate_seq_config(ctypes.byref(cfg))


# ---- checks ------------------------------------------------------------------
# The checks run before every launch, so the common case is one expression per
# tensor; what is wrong is looked up only where something is.

def _refuse(what, cfg, name, t, dtype, shape, device):
    st = validate_seq(cfg)
    if st != 0:
        raise Pack3DError(st, what)
    if t.dtype != dtype:
        raise ValueError(f"{what}: {name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: {name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what}: {name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{what}: {name} is on {t.device}, other tensors on {device}")
    raise ValueError(f"{what}: {name} must be contiguous")


def _require(what, cfg, name, t, dtype, shape, device):
    """Refuses, before anything runs, a tensor that is not what the kernels will take it for."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device.index or not t.is_contiguous():
        _refuse(what, cfg, name, t, dtype, shape, device)


_modules = []


def _torch():
    if not _modules:       # torch is imported with the first call, not with the package
        import torch
        _modules.append((torch, {BF16: torch.bfloat16, F32: torch.float32}))
    return _modules[0]


_templates = {}


def _new(device, dtype, *shape):
    """torch.empty, from an empty tensor of the device and type: it takes half as long as naming both.  Only a plain
    tensor is kept for it: under FakeTensorMode and the like torch.empty gives something else."""
    key = device.index, dtype
    t = _templates.get(key)
    if t is None:
        torch = _torch()[0]
        t = torch.empty(0, dtype=dtype, device=device)
        if type(t) is torch.Tensor:
            _templates[key] = t
    return t.new_empty(*shape)


def _check_err_word(what, err, device, torch):
    if err is not None and (err.dtype != torch.int32 or err.numel() < 1 or err.device != device):
        raise ValueError(f"{what}: the error word must be an int32 tensor of at least one element on {device}")


def _check_workspace(what, workspace, device):
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"{what}: the workspace must be a contiguous tensor on {device}")


def _owned(what, *tensors):
    if any(t is None for t in tensors):
        raise ValueError(f"{what}: with an explicit stream, give every output and the workspace too")


def _p(t):
    return None if t is None else t.data_ptr()


def _raw_stream(device):
    """The device's current stream as the handle the C ABI takes.  (torch.cuda.current_stream builds an object for
    it, which takes longer than the launch itself of a small call.)"""
    return _modules[0][0]._C._cuda_getCurrentRawStream(device.index)


def _run(torch, fn, device, stream, *args):
    """Runs a C entry point on `stream` (the device's current one by default) with the tensors' device current, and
    returns its status."""
    if stream is None:
        stream = _raw_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        return fn(*args, stream)
    with torch.cuda.device(device):
        return fn(*args, stream)


def _call(torch, what, fn, device, stream, *args):
    st = _run(torch, fn, device, stream, *args)
    if st != 0:
        raise Pack3DError(st, what)


def _window_args(what, cfg, q, k, v, cu_q, cu_k):
    torch, types = _torch()
    if q.dim() != 3 or k.dim() != 3 or cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError(f"{what}: q and k are [rows, heads, {DH}], cu_q is [batch + 1]")
    T, dev = types.get(cfg.dtype), q.device
    keys = (k.shape[0], cfg.Hkv, DH)
    if not q.is_cuda:
        _refuse(what, cfg, "q", q, T, (q.shape[0], cfg.Hq, DH), dev)
    _require(what, cfg, "q", q, T, (q.shape[0], cfg.Hq, DH), dev)
    _require(what, cfg, "k", k, T, keys, dev)
    _require(what, cfg, "v", v, T, keys, dev)
    _require(what, cfg, "cu_q", cu_q, torch.int32, cu_q.shape, dev)
    if cu_k is not cu_q:
        _require(what, cfg, "cu_k", cu_k, torch.int32, cu_q.shape, dev)
    return torch, T, dev


# ---- windowed attention ------------------------------------------------------------

def window_attn(cfg: SeqConfig, q, k, v, cu_q, cu_k=None, out=None, lse=None, err=None, stream=None):
    """pack3d_window_attn: returns (out like q, lse float [rows, Hq]), into the given tensors where there are any.
    cu_k defaults to cu_q.  Rows of no sequence are 0 (lse -infinity) in tensors made here and stay as they were in
    given ones; give both or none."""
    what = "pack3d_window_attn"
    cu_k = cu_q if cu_k is None else cu_k
    torch, T, dev = _window_args(what, cfg, q, k, v, cu_q, cu_k)
    if stream is not None:
        _owned(what, out, lse)
    if (out is None) != (lse is None):
        raise ValueError(f"{what}: give both out and lse or none of them")
    new = out is None
    if new:
        out = torch.empty_like(q)
        lse = _new(dev, torch.float32, q.shape[0], cfg.Hq)
        if cu_q.shape[0] == 1:     # no sequence at all: nothing is launched
            return out.zero_(), lse.fill_(-math.inf)
    else:
        _require(what, cfg, "out", out, T, tuple(q.shape), dev)
        _require(what, cfg, "lse", lse, torch.float32, tuple(q.shape[:2]), dev)
    _check_err_word(what, err, dev, torch)
    _call(torch, what, lib.pack3d_window_attn, dev, stream, ctypes.byref(cfg), cu_q.shape[0] - 1, q.shape[0],
          k.shape[0], cu_q.data_ptr(), cu_k.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          lse.data_ptr(), int(new), _p(err))
    return out, lse


def window_attn_bwd_workspace_bytes(cfg: SeqConfig, batch: int, q_rows: int, k_rows: int) -> int:
    return int(lib.pack3d_window_attn_bwd_workspace_bytes(ctypes.byref(cfg), batch, q_rows, k_rows))


def window_attn_bwd(cfg: SeqConfig, q, k, v, cu_q, cu_k, out, lse, dout, dq=None, dk=None, dv=None, workspace=None,
                    err=None, stream=None):
    """pack3d_window_attn_bwd: returns (dq, dk, dv) of <dout, out>, from window_attn's out and lse.  Rows of no
    sequence are 0 in gradients made here and stay as they were in given ones; give all three or none."""
    what = "pack3d_window_attn_bwd"
    cu_k = cu_q if cu_k is None else cu_k
    torch, T, dev = _window_args(what, cfg, q, k, v, cu_q, cu_k)
    if stream is not None:
        _owned(what, dq, dk, dv, workspace)
    shape = q.shape
    _require(what, cfg, "out", out, T, shape, dev)
    _require(what, cfg, "dout", dout, T, shape, dev)
    _require(what, cfg, "lse", lse, torch.float32, shape[:2], dev)
    new = dq is None
    if (dk is None) != new or (dv is None) != new:
        raise ValueError(f"{what}: give all of dq, dk and dv or none of them")
    if not new:
        for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            _require(what, cfg, name, t, T, tuple(like.shape), dev)
    if workspace is not None:
        _check_workspace(what, workspace, dev)
    _check_err_word(what, err, dev, torch)
    if new:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        if cu_q.shape[0] == 1:     # no sequence at all: nothing is launched
            return dq.zero_(), dk.zero_(), dv.zero_()
    batch, q_rows, k_rows = cu_q.shape[0] - 1, q.shape[0], k.shape[0]
    if workspace is None:
        n = window_attn_bwd_workspace_bytes(cfg, batch, q_rows, k_rows)
        workspace = _new(dev, torch.uint8, max(n, 256))
    else:
        n = workspace.numel() * workspace.element_size()
    _call(torch, what, lib.pack3d_window_attn_bwd, dev, stream, ctypes.byref(cfg), batch, q_rows, k_rows,
          cu_q.data_ptr(), cu_k.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
          dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), int(new), workspace.data_ptr(), n, _p(err))
    return dq, dk, dv


def window_attention(cfg: SeqConfig, q, k, v, cu_q, cu_k=None, err=None):
    """pack3d_window_attn as a differentiable PyTorch op: returns out, with gradients of q, k and v by
    pack3d_window_attn_bwd.  Neither direction synchronises; both can be captured into a CUDA graph, as long as no
    eager autograd graph of the same leaves is alive then (PyTorch's gradient accumulation would wait for that
    graph's stream, which ends the capture with an error; detached copies of the leaves have none)."""
    return _autograd().apply(cfg, q, k, v, cu_q, cu_q if cu_k is None else cu_k, err)


_autograd_class = None


def _autograd():
    global _autograd_class
    if _autograd_class is None:
        import torch
        from torch.autograd.function import once_differentiable

        class WindowAttention(torch.autograd.Function):
            @staticmethod
            def forward(ctx, cfg, q, k, v, cu_q, cu_k, err):
                out, lse = window_attn(cfg, q, k, v, cu_q, cu_k, err=err)
                ctx.cfg = SeqConfig.from_buffer_copy(cfg)
                ctx.err = err
                ctx.save_for_backward(q, k, v, cu_q, cu_k, out, lse)
                return out

            @staticmethod
            @once_differentiable
            def backward(ctx, dout):
                # Saved-tensor hooks may give back other tensors than the forward saved: of equal values but other
                # strides, which is put right here, or of another type or device, which the call refuses.
                saved = [t.contiguous() for t in ctx.saved_tensors]
                if dout.dtype is not saved[0].dtype:
                    dout = dout.to(saved[0].dtype)
                return None, *window_attn_bwd(ctx.cfg, *saved, dout.contiguous(), err=ctx.err), None, None, None

        _autograd_class = WindowAttention
    return _autograd_class


# ---- the paged cache ------------------------------------------------------------------

def _cache_args(what, cfg, k_pages, v_pages, table, lengths):
    torch, types = _torch()
    if k_pages.dim() != 4 or table.dim() != 2:
        raise ValueError(f"{what}: the pages are [num_pages, page, Hkv, {DH}], the table is [batch, max_pages]")
    T, dev = types.get(cfg.dtype), k_pages.device
    shape = (k_pages.shape[0], cfg.page, cfg.Hkv, DH)
    if not k_pages.is_cuda:
        _refuse(what, cfg, "k_pages", k_pages, T, shape, dev)
    _require(what, cfg, "k_pages", k_pages, T, shape, dev)
    _require(what, cfg, "v_pages", v_pages, T, shape, dev)
    _require(what, cfg, "table", table, torch.int32, table.shape, dev)
    _require(what, cfg, "lengths", lengths, torch.int32, (table.shape[0],), dev)
    return torch, T, dev


def cache_append(cfg: SeqConfig, k, v, k_pages, v_pages, table, lengths, cu=None, err=None, stream=None):
    """pack3d_cache_append: the rows of k and v [rows, Hkv, 64] into the slots behind `lengths` (which is not
    changed); cu int32 [batch + 1], or None for one row per sequence."""
    what = "pack3d_cache_append"
    torch, T, dev = _cache_args(what, cfg, k_pages, v_pages, table, lengths)
    rows = k.shape[0]
    _require(what, cfg, "k", k, T, (rows, cfg.Hkv, DH), dev)
    _require(what, cfg, "v", v, T, (rows, cfg.Hkv, DH), dev)
    if cu is not None:
        _require(what, cfg, "cu", cu, torch.int32, (table.shape[0] + 1,), dev)
    _check_err_word(what, err, dev, torch)
    _call(torch, what, lib.pack3d_cache_append, dev, stream, ctypes.byref(cfg), table.shape[0], rows, _p(cu),
          lengths.data_ptr(), table.data_ptr(), table.shape[1], k_pages.shape[0], k.data_ptr(), v.data_ptr(),
          k_pages.data_ptr(), v_pages.data_ptr(), _p(err))


def cache_attn_workspace_bytes(cfg: SeqConfig, batch: int, max_pages: int, with_weights: bool = False) -> int:
    return int(lib.pack3d_cache_attn_workspace_bytes(ctypes.byref(cfg), batch, max_pages, int(with_weights)))


def cache_attn(cfg: SeqConfig, q, k_pages, v_pages, table, lengths, out=None, lse=None, weights=None,
               accumulate: bool = False, workspace=None, err=None, stream=None):
    """pack3d_cache_attn: attention of one new token per sequence, q [batch, Hq, 64], over the cache.  Returns
    (out like q, lse float [batch, Hq]); `weights` float [batch, max_pages * page] gets the token's attention weights
    (added to what it holds with `accumulate`)."""
    what = "pack3d_cache_attn"
    torch, T, dev = _cache_args(what, cfg, k_pages, v_pages, table, lengths)
    batch, max_pages = table.shape
    _require(what, cfg, "q", q, T, (batch, cfg.Hq, DH), dev)
    if stream is not None:
        _owned(what, out, lse)
        if workspace is None and cache_attn_workspace_bytes(cfg, batch, max_pages, weights is not None):
            _owned(what, workspace)
    if out is None:
        out = torch.empty_like(q)
    else:
        _require(what, cfg, "out", out, T, tuple(q.shape), dev)
    if lse is None:
        lse = _new(dev, torch.float32, batch, cfg.Hq)
    else:
        _require(what, cfg, "lse", lse, torch.float32, (batch, cfg.Hq), dev)
    if weights is not None:
        _require(what, cfg, "weights", weights, torch.float32, (batch, max_pages * cfg.page), dev)
    n = 0
    if workspace is not None:
        _check_workspace(what, workspace, dev)
        n = workspace.numel() * workspace.element_size()
    elif weights is not None and batch:                # always needs one
        n = cache_attn_workspace_bytes(cfg, batch, max_pages, True)
        workspace = _new(dev, torch.uint8, n)
    _check_err_word(what, err, dev, torch)
    args = (ctypes.byref(cfg), batch, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(),
            max_pages, k_pages.shape[0], lengths.data_ptr(), out.data_ptr(), lse.data_ptr(), _p(weights),
            int(bool(accumulate)))
    st = _run(torch, lib.pack3d_cache_attn, dev, stream, *args, _p(workspace), n, _p(err))
    if st == ERR_WORKSPACE and workspace is None:      # short calls need none: asked for only when missed
        n = cache_attn_workspace_bytes(cfg, batch, max_pages, weights is not None)
        workspace = _new(dev, torch.uint8, n)
        st = _run(torch, lib.pack3d_cache_attn, dev, stream, *args, workspace.data_ptr(), n, _p(err))
    if st != 0:
        raise Pack3DError(st, what)
    return out, lse


def cache_evict(cfg: SeqConfig, k_pages, v_pages, table, lengths, weights, new_table, budget: int, recent: int,
                kept=None, new_weights=None, new_lengths=None, err=None, stream=None):
    """pack3d_cache_evict: every sequence cut to `budget` slots, copied to the pages of new_table int32 [batch,
    new_max_pages].  Returns (kept int32 [batch, budget], new_weights float [batch, new_max_pages * page],
    new_lengths int32 [batch])."""
    what = "pack3d_cache_evict"
    torch, T, dev = _cache_args(what, cfg, k_pages, v_pages, table, lengths)
    batch, max_pages = table.shape
    _require(what, cfg, "weights", weights, torch.float32, (batch, max_pages * cfg.page), dev)
    if new_table.dim() != 2:
        raise ValueError(f"{what}: new_table is [batch, new_max_pages]")
    _require(what, cfg, "new_table", new_table, torch.int32, (batch, new_table.shape[1]), dev)
    if stream is not None:
        _owned(what, kept, new_weights, new_lengths)
    shapes = ((batch, max(int(budget), 0)), (batch, new_table.shape[1] * cfg.page), (batch,))
    outs = []
    for name, t, dt, shape in (("kept", kept, torch.int32, shapes[0]), ("new_weights", new_weights, torch.float32,
                               shapes[1]), ("new_lengths", new_lengths, torch.int32, shapes[2])):
        if t is None:
            t = _new(dev, dt, *shape)
        else:
            _require(what, cfg, name, t, dt, shape, dev)
        outs.append(t)
    _check_err_word(what, err, dev, torch)
    _call(torch, what, lib.pack3d_cache_evict, dev, stream, ctypes.byref(cfg), batch, k_pages.data_ptr(),
          v_pages.data_ptr(), k_pages.shape[0], table.data_ptr(), max_pages, lengths.data_ptr(), weights.data_ptr(),
          int(budget), int(recent), new_table.data_ptr(), new_table.shape[1], outs[0].data_ptr(), outs[1].data_ptr(),
          outs[2].data_ptr(), _p(err))
    return tuple(outs)


class PagedCache:
    """Pages, table, lengths and error word of one batch of sequences on one device, and the calls on them.

    Every sequence owns the pages of `capacity` slots.  With a `budget` (evict's), attend collects the attention
    weights and every sequence owns the pages of `budget` further slots, which evict fills and exchanges for the old
    ones.  No two rows of the table name the same page, and evict relies on that.  Rows beyond the capacity are not
    written and set the error that check() raises.  Nothing here waits for the device; check() does."""

    def __init__(self, cfg: SeqConfig, batch: int, capacity: int, budget: int = 0, device="cuda"):
        st = validate_seq(cfg)
        if st != 0:
            raise Pack3DError(st, "PagedCache")
        torch, types = _torch()
        T = types[cfg.dtype]
        if batch < 1 or capacity < 1 or budget < 0 or budget > capacity:
            raise ValueError("PagedCache: batch and capacity are at least 1, the budget is at most the capacity")
        self.cfg, self.budget = cfg, budget
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"PagedCache: lives on a CUDA device, not on {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        wide, spare = -(-capacity // cfg.page), -(-budget // cfg.page)
        pages = torch.arange(batch * (wide + spare), dtype=torch.int32, device=dev)
        self.table = pages[:batch * wide].view(batch, wide).clone()
        self.spare = pages[batch * wide:].view(batch, spare).clone()
        shape = (batch * (wide + spare), cfg.page, cfg.Hkv, DH)
        self.k_pages = torch.empty(shape, dtype=T, device=dev)
        self.v_pages = torch.empty(shape, dtype=T, device=dev)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.weights = torch.zeros((batch, wide * cfg.page), device=dev) if budget else None
        self.err = torch.zeros(4, dtype=torch.int32, device=dev)

    def append(self, k, v, cu=None):
        """New rows behind the cached ones: one per sequence, or cu's."""
        cache_append(self.cfg, k, v, self.k_pages, self.v_pages, self.table, self.lengths, cu, err=self.err)
        self.lengths += 1 if cu is None else cu.diff()

    def attend(self, q, out=None):
        """Attention of the newest token of every sequence (appended before)."""
        return cache_attn(self.cfg, q, self.k_pages, self.v_pages, self.table, self.lengths, out=out,
                          weights=self.weights, accumulate=True, err=self.err)[0]

    def evict(self, recent: int):
        """Cuts every sequence to the budget; returns the old slots that stay, int32 [batch, budget], -1 behind."""
        if not self.budget:
            raise ValueError("PagedCache: made without a budget")
        kept, weights, lengths = cache_evict(self.cfg, self.k_pages, self.v_pages, self.table, self.lengths,
                                             self.weights, self.spare, self.budget, recent, err=self.err)
        n = self.spare.shape[1]
        old = self.table[:, :n].clone()
        self.table[:, :n] = self.spare
        self.spare.copy_(old)
        self.weights.zero_()
        self.weights[:, :weights.shape[1]] = weights
        self.lengths.copy_(lengths)
        return kept

    def check(self):
        with _torch()[0].cuda.device(self.err.device):
            st = check_status(self.err)
        if st != 0:
            raise Pack3DError(st, "PagedCache")
