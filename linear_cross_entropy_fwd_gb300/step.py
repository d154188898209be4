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

from . import (_check, _check_out, _dtype_code, _is32, load_library, make_opts,
               scale_convert)


def _call(fn, dev, dtype, args, *, sync, workspace, info, ids32=0):
    """Run C entry ``fn(*args, opts)`` on ``dev``'s current stream."""
    o = make_opts(dtype, torch.cuda.current_stream(dev).cuda_stream, sync=1 if sync else 0,
                  target_is_int32=ids32)
    if workspace is not None:
        _check_out(workspace, (workspace.numel(),), workspace.dtype, dev, "workspace")
        o.workspace = workspace.data_ptr()
        o.workspace_bytes = workspace.numel() * workspace.element_size()
    if info is not None:
        status = torch.zeros((), dtype=torch.int32, device=dev)
        used = ctypes.c_size_t(0)
        o.status_dev = status.data_ptr()
        o.workspace_used = ctypes.pointer(used)
    if dev.index == torch.cuda.current_device():
        st = fn(*args, ctypes.byref(o))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, ctypes.byref(o))
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
    lib = load_library()
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
    times the sum of ``dY[i]`` over the tokens with ``ids[i] == v``, added in
    ascending i.  ``accumulate=True`` adds it to ``dW`` (a weight tied to the
    head's) and touches no other row; otherwise dW is overwritten."""
    lib = load_library()
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
