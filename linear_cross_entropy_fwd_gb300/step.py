"""Binding of the operators around the head: embedding lookup and its gradient,
attention over packed sequences, and Newton-Schulz orthogonalisation.

As in the package's root module this is argument marshalling only.  Each call
runs on the current CUDA stream with its input's device current.  With
``sync=True`` it blocks and kernel-side errors raise ``FlceError``; otherwise
``info['status']`` (a 0-d int32 device tensor, filled in when a dict is given
as ``info``) holds the status once the stream has reached it.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import (FLCE_FP32, FlceAttn, FlceOpts, _check, _check_out, _dtype_code, _is32,
               load_library, make_opts, scale_convert)


_lib = None
_defaults = None  # a flce_opts as flce_opts_init leaves it, with sync off


def _library():
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


def _call(fn, dev, dtype, args, *, sync, workspace, info, ids32=0):
    """Run C entry ``fn(*args, opts)`` on ``dev``'s current stream."""
    global _defaults
    if _defaults is None:
        _defaults = bytes(make_opts(sync=0))
    o = FlceOpts.from_buffer_copy(_defaults)
    if dtype is torch.float32:
        o.dtype = FLCE_FP32
    index = dev.index
    o.stream = torch._C._cuda_getCurrentRawStream(index)
    if sync:
        o.sync = 1
    if ids32:
        o.target_is_int32 = 1
    if workspace is not None:
        _check_out(workspace, (workspace.numel(),), workspace.dtype, dev, "workspace")
        o.workspace = workspace.data_ptr()
        o.workspace_bytes = workspace.numel() * workspace.element_size()
    if info is not None:
        status = torch.zeros((), dtype=torch.int32, device=dev)
        used = ctypes.c_size_t(0)
        o.status_dev = status.data_ptr()
        o.workspace_used = ctypes.pointer(used)
    if index == torch.cuda.current_device():
        st = fn(*args, ctypes.byref(o))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, ctypes.byref(o))
    if st:
        _check(st)
    if info is not None:
        info.update(status=status, workspace_bytes=used.value)


def _check_ids(ids: torch.Tensor, N: int | None, device) -> None:
    if ids.dim() != 1 or (N is not None and ids.shape[0] != N):
        raise ValueError("ids must be a vector with one id per row")
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError("ids must be int64 or int32")
    if not ids.is_cuda or ids.device != device or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous CUDA tensor on {device}")


def flce_embed_fwd(W: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
                   ignore_index: int = -100, out: torch.Tensor | None = None,
                   sync: bool = False, info: dict | None = None) -> torch.Tensor:
    """``out[i] = scale * W[ids[i]]`` in W's dtype (bf16 or fp32); rows of zeros
    where ``ids[i]`` is ``ignore_index``.  W [V, H], ids [N]; returns [N, H]."""
    lib = _library()
    if W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous CUDA tensor [V, H]")
    _dtype_code(W)
    V, H = W.shape
    _check_ids(ids, None, W.device)
    N = ids.shape[0]
    if out is None:
        out = torch.empty((N, H), dtype=W.dtype, device=W.device)
    else:
        _check_out(out, (N, H), W.dtype, W.device, "out")
    _call(lib.flce_embed_fwd, W.device, W.dtype,
          (W.data_ptr(), ids.data_ptr(), N, H, V, float(scale), int(ignore_index),
           out.data_ptr()), sync=sync, workspace=None, info=info, ids32=_is32(ids))
    return out


def flce_embed_bwd(dY: torch.Tensor, ids: torch.Tensor, V: int | None = None, *,
                   scale: float = 1.0, ignore_index: int = -100,
                   dW: torch.Tensor | None = None, accumulate: bool = False,
                   sync: bool = False, workspace: torch.Tensor | None = None,
                   info: dict | None = None) -> torch.Tensor:
    """The gradient of ``flce_embed_fwd`` in fp32 [V, H]: row v is ``scale``
    times the sum of ``dY[i]`` over the tokens with ``ids[i] == v``, added in a
    fixed order.  ``accumulate=True`` adds it to ``dW`` (a weight tied to the
    head's) and touches no other row; otherwise dW is overwritten."""
    lib = _library()
    if dY.dim() != 2 or not dY.is_cuda or not dY.is_contiguous():
        raise ValueError("dY must be a contiguous CUDA tensor [N, H]")
    _dtype_code(dY)
    N, H = dY.shape
    _check_ids(ids, N, dY.device)
    if dW is None:
        if V is None or accumulate:
            raise ValueError("give V, or dW to accumulate into")
        dW = torch.empty((int(V), H), dtype=torch.float32, device=dY.device)
    V = dW.shape[0] if V is None else int(V)
    _check_out(dW, (V, H), torch.float32, dY.device, "dW")
    _call(lib.flce_embed_bwd, dY.device, dY.dtype,
          (dY.data_ptr(), ids.data_ptr(), N, H, V, float(scale), int(ignore_index),
           dW.data_ptr(), 1 if accumulate else 0),
          sync=sync, workspace=workspace, info=info, ids32=_is32(ids))
    return dW


class _EmbedFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, ignore_index):
        ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.args = (weight.shape[0], weight.dtype, scale, ignore_index)
        return flce_embed_fwd(weight.contiguous(), ids, scale=scale, ignore_index=ignore_index)

    @staticmethod
    @once_differentiable  # the kernels' results carry no graph of their own
    def backward(ctx, grad_out):
        (ids,) = ctx.saved_tensors
        V, dtype, scale, ignore_index = ctx.args
        dW = flce_embed_bwd(grad_out.contiguous(), ids, V, scale=scale,
                            ignore_index=ignore_index)
        if dtype != torch.float32:
            dW = scale_convert(dW, torch.empty(dW.shape, dtype=dtype, device=dW.device))
        return dW, None, None, None


class Embedding(torch.nn.Module):
    """``embed(weight, ids)`` -> [N, H]; the gradient comes back in the weight's dtype."""

    def __init__(self, scale: float = 1.0, ignore_index: int = -100):
        super().__init__()
        self.scale = scale
        self.ignore_index = ignore_index

    def forward(self, weight, ids):
        return _EmbedFunction.apply(weight, ids, self.scale, self.ignore_index)


def _heads_tensor(name, t, T, heads, D, device):
    """A bf16 [T, heads, D] tensor with a contiguous last axis on ``device``;
    returns its address and its token and head strides."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bf16, got {t.dtype}")
    if t.shape != (T, heads, D):
        raise ValueError(f"{name} must have shape {(T, heads, D)}, got {tuple(t.shape)}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    token, head, last = t.stride()
    if last != 1 and D > 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    return t.data_ptr(), token, head


def _attn_args(q, k, v, cu_seqlens, scale, o, lse):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q [T, heads_q, D], k and v [T, heads_kv, D]")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    dev = q.device
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold one offset more than there are sequences")
    for name, t, shape, dtype in (("lse", lse, (Hq, T), torch.float32),
                                  ("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32)):
        if t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
            _check_out(t, shape, dtype, dev, name)
    # in the order of the structure's fields
    return FlceAttn(T, cu_seqlens.shape[0] - 1, cu_seqlens.data_ptr(), Hq, Hkv, D,
                    D ** -0.5 if scale is None else float(scale),
                    *_heads_tensor("q", q, T, Hq, D, dev), *_heads_tensor("k", k, T, Hkv, D, dev),
                    *_heads_tensor("v", v, T, Hkv, D, dev), *_heads_tensor("o", o, T, Hq, D, dev),
                    lse.data_ptr())


def flce_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
                  scale: float | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, sync: bool = False,
                  workspace: torch.Tensor | None = None, info: dict | None = None):
    """Causal attention over packed sequences; returns (o, lse).

    q [T, heads_q, D], k and v [T, heads_kv, D] in bf16 with a contiguous last
    axis (slices of one projection's output will do), none of it over ``out``;
    ``cu_seqlens`` int32 [sequences + 1] on the device.  ``scale`` defaults to D ** -0.5.  o is
    [T, heads_q, D], lse fp32 [heads_q, T]."""
    lib = _library()
    if q.dim() != 3:
        raise ValueError("q [T, heads_q, D], k and v [T, heads_kv, D]")
    T, Hq, D = q.shape
    dev = q.device
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    a = _attn_args(q, k, v, cu_seqlens, scale, out, lse)
    _call(lib.flce_attn_fwd, dev, q.dtype, (ctypes.byref(a),), sync=sync,
          workspace=workspace, info=info)
    return out, lse


def flce_attn_bwd(dO: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  o: torch.Tensor, lse: torch.Tensor, cu_seqlens: torch.Tensor, *,
                  scale: float | None = None, dq: torch.Tensor | None = None,
                  dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                  sync: bool = False, workspace: torch.Tensor | None = None,
                  info: dict | None = None):
    """Gradients of ``flce_attn_fwd`` at its inputs and outputs; returns
    (dq, dk, dv) in bf16, dk and dv summed over the query heads they serve.  They may
    share memory with ``o``, but not with the other inputs or one another."""
    lib = _library()
    a = _attn_args(q, k, v, cu_seqlens, scale, o, lse)
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=k.dtype, device=k.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=v.dtype, device=v.device) if dv is None else dv
    for name, t, like in (("dO", dO, q), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        at, token, head = _heads_tensor(name, t, *like.shape, q.device)
        setattr(a, name, at)
        setattr(a, name + "_token", token)
        setattr(a, name + "_head", head)
    _call(lib.flce_attn_bwd, q.device, q.dtype, (ctypes.byref(a),), sync=sync,
          workspace=workspace, info=info)
    return dq, dk, dv


def _strided(t):
    """t itself if the library takes its strides, else a contiguous copy (a
    broadcast axis has stride 0)."""
    ok = (t.stride(2) == 1 and all(s > 0 and s % 8 == 0 for s in t.stride()[:2])
          and t.data_ptr() % 16 == 0)
    return t if ok else t.contiguous()


class _AttnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, scale):
        q, k, v = _strided(q), _strided(k), _strided(v)
        o, lse = flce_attn_fwd(q, k, v, cu_seqlens, scale=scale)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.scale = scale
        return o

    @staticmethod
    @once_differentiable  # the kernels' results carry no graph of their own
    def backward(ctx, grad_out):
        q, k, v, o, lse, cu_seqlens = ctx.saved_tensors
        dq, dk, dv = flce_attn_bwd(_strided(grad_out), q, k, v, o, lse, cu_seqlens,
                                   scale=ctx.scale)
        return dq, dk, dv, None, None


class PackedAttention(torch.nn.Module):
    """``attn(q, k, v, cu_seqlens)`` -> o, differentiable in q, k and v."""

    def __init__(self, scale: float | None = None):
        super().__init__()
        self.scale = scale

    def forward(self, q, k, v, cu_seqlens):
        return _AttnFunction.apply(q, k, v, cu_seqlens, self.scale)


def flce_orthogonalize(G: torch.Tensor, *, steps: int = 5,
                       coeffs: tuple[float, float, float] = (3.4445, -4.7750, 2.0315),
                       eps: float = 1e-7, out: torch.Tensor | None = None, sync: bool = False,
                       workspace: torch.Tensor | None = None, info: dict | None = None):
    """Newton-Schulz orthogonalisation of each matrix of G [..., rows, cols]
    (bf16 or fp32): ``X = G / (|G|_F + eps)``, then ``steps`` times
    ``X = a X + (b A + c A A) X`` with ``A = X X^T``.  Returns X in bf16."""
    lib = _library()
    if G.dim() < 2 or not G.is_cuda or not G.is_contiguous():
        raise ValueError("G must be a contiguous CUDA tensor [..., rows, cols]")
    _dtype_code(G)
    if len(coeffs) != 3:
        raise ValueError("coeffs must be (a, b, c)")
    rows, cols = G.shape[-2:]
    batch = 1
    for n in G.shape[:-2]:
        batch *= n
    if out is None:
        out = torch.empty(G.shape, dtype=torch.bfloat16, device=G.device)
    else:
        _check_out(out, G.shape, torch.bfloat16, G.device, "out")
    abc = (ctypes.c_float * 3)(*coeffs)
    _call(lib.flce_orthogonalize, G.device, G.dtype,
          (G.data_ptr(), batch, rows, cols, int(steps), ctypes.cast(abc, ctypes.c_void_p),
           float(eps), out.data_ptr()), sync=sync, workspace=workspace, info=info)
    return out
