"""Binding of the operators between a model's blocks: the residual join with its norms and
gate, and activation checkpoints in 8 bits with the weight gradient that reads them.

Conventions as in ``step.py``: argument marshalling only, the current CUDA stream, errors
through ``sync=True`` or ``info['status']``.
"""
from __future__ import annotations

import math
import struct
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _check_out, _dtype_code, scale_convert
from .step import _call, _library

NORMS = {"rms": 0, "layer": 1}
ACTS = {None: 0, "none": 0, "sigmoid": 1, "tanh": 2}
GATE_NONE, GATE_SCALAR, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = range(5)
_HALF = (torch.bfloat16, torch.float32)


# struct flce_resnorm, for _pack: at the size of these calls, filling a ctypes structure
# field by field takes longer than the library's side of the call.
_pack = struct.Struct("@qq7i3f" + "Pq" * 3 + "4P" + "Pq" + "P" + "Pq" + "P" + "Pq" * 5 + "4P").pack
assert struct.calcsize("@qq7i3f") % 8 == 0
_NONE = (0, 0)


def _rows(name, t, shape, dtype, device):
    """A [N, H] tensor of ``dtype`` with a contiguous last axis; its address and row stride."""
    if t is None:
        return _NONE
    row, last = t.stride() if t.dim() == 2 else (0, 0)
    if t.dtype is dtype and t.shape == shape and t.device == device and last == 1:
        return t.data_ptr(), row
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if last != 1 and t.numel():  # (without rows its strides are anything)
        raise ValueError(f"{name} must have a contiguous last axis")
    return t.data_ptr(), row


def _vector(name, t, shape, dtype, device):
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _check_out(t, shape, dtype, device, name)
    return t.data_ptr()


def _gate_kind(gate, N, H):
    """A scalar or [H] is a learned gate; [N, 1] and [N, H] are gates computed per token."""
    if gate.dim() < 2:
        if gate.dim() == 1 and gate.shape[0] != H:
            raise ValueError(f"gate must have {H} elements, got {gate.shape[0]}")
        return GATE_CHANNEL if gate.dim() else GATE_SCALAR
    if gate.dim() != 2 or gate.shape[0] != N or gate.shape[1] not in (1, H):
        raise ValueError(f"gate must be a scalar, ({H},), ({N}, 1) or ({N}, {H}), "
                         f"got {tuple(gate.shape)}")
    # of H = 1 there is no such tensor: H is at least 8
    return GATE_FULL if gate.shape[1] == H else GATE_TOKEN


def _gate_address(gate, kind, shape, dtype, device):
    if kind == GATE_FULL:
        return _rows("gate", gate, shape, dtype, device)
    if gate.dtype is not dtype:
        raise TypeError(f"gate must be {dtype}, got {gate.dtype}")
    if gate.device != device or (kind == GATE_CHANNEL and not gate.is_contiguous()):
        raise ValueError(f"gate must be a contiguous CUDA tensor on {device}")
    return gate.data_ptr(), gate.stride(0) if kind == GATE_TOKEN else 0


def _common(dt, shape, dev, stream_dtype, w_post, b_post, w_pre, b_pre, gate, gate_act, kind,
            alpha, beta, eps, post_norm, pre_norm):
    """The fields that both passes share: the structure's up to ``eps``, the gate's, the
    parameters'; and the gate's kind."""
    if kind not in NORMS:
        raise ValueError(f"kind must be one of {sorted(NORMS)}")
    if gate_act not in ACTS:
        raise ValueError(f"gate_act must be one of {[k for k in ACTS if k]}")
    if stream_dtype is not dt and stream_dtype is not torch.float32:
        raise TypeError(f"the stream must be {dt} or fp32")
    given = w_post is not None or b_post is not None
    post = given if post_norm is None else bool(post_norm)
    if given and not post:
        raise ValueError("w_post and b_post need post_norm")
    if not pre_norm and (w_pre is not None or b_pre is not None):
        raise ValueError("w_pre and b_pre need pre_norm")
    N, H = shape
    gk = GATE_NONE if gate is None else _gate_kind(gate, N, H)
    learned = gate if gk == GATE_SCALAR or gk == GATE_CHANNEL else None
    # the one type of all parameters: y's, or fp32
    pt = None
    for t in (w_post, b_post, w_pre, b_pre, learned):
        if t is not None:
            if pt is None:
                pt = t.dtype
            if t.dtype is not pt or (pt is not dt and pt is not torch.float32):
                raise TypeError(f"weights, biases and learned gates must all be {dt} or all fp32")
    head = (N, H, NORMS[kind], post, bool(pre_norm), stream_dtype is torch.float32,
            pt is torch.float32, gk, ACTS[gate_act], alpha, beta, eps)
    ga = _NONE if gate is None else _gate_address(gate, gk, shape, dt if learned is None else pt,
                                                  dev)
    one = (H,)
    vecs = (_vector("w_post", w_post, one, pt, dev), _vector("b_post", b_post, one, pt, dev),
            _vector("w_pre", w_pre, one, pt, dev), _vector("b_pre", b_pre, one, pt, dev))
    return head, ga, vecs, gk


def _check_stats(stats, N, dev):
    if stats.shape != (4, N) or stats.dtype is not torch.float32 or stats.device != dev \
            or not stats.is_contiguous():
        _check_out(stats, (4, N), torch.float32, dev, "stats")
    return stats.data_ptr()


def _check_y(y, name="y"):
    if y.dim() != 2 or not y.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [N, H]")
    _dtype_code(y)


class Checkpoint:
    """Activations [N, H] in 8 bits: ``data`` holds e4m3 codes and a power of two for every 32
    of a row, in the layout that ``include/flce.h`` gives (``flce_ckpt_bytes(N, H)`` bytes)."""

    __slots__ = ("data", "N", "H")

    def __init__(self, data: torch.Tensor, N: int, H: int):
        if data.dtype is not torch.uint8 or not data.is_cuda or not data.is_contiguous():
            raise ValueError("data must be a contiguous uint8 CUDA tensor")
        if data.numel() != checkpoint_bytes(N, H):
            raise ValueError(f"a checkpoint of {(N, H)} has {checkpoint_bytes(N, H)} bytes, "
                             f"got {data.numel()}")
        self.data, self.N, self.H = data, N, H

    @classmethod
    def empty(cls, N: int, H: int, device) -> "Checkpoint":
        return cls(torch.empty(checkpoint_bytes(N, H), dtype=torch.uint8, device=device), N, H)


def checkpoint_bytes(N: int, H: int) -> int:
    """Bytes of a checkpoint of [N, H]."""
    n = _library().flce_ckpt_bytes(N, H)
    if n == 0 and N != 0:
        raise ValueError(f"no checkpoint has the shape {(N, H)}")
    return n


def flce_resnorm_fwd(y: torch.Tensor, h: torch.Tensor | None = None, *,
                     w_pre: torch.Tensor | None = None, b_pre: torch.Tensor | None = None,
                     w_post: torch.Tensor | None = None, b_post: torch.Tensor | None = None,
                     gate: torch.Tensor | None = None, gate_act: str | None = None,
                     kind: str = "rms", alpha: float = 1.0, beta: float = 1.0,
                     eps: float = 1e-6, pre_norm: bool = True, post_norm: bool | None = None,
                     stream_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                     z: torch.Tensor | None = None, stats: torch.Tensor | None = None,
                     checkpoint: Checkpoint | None = None, sync: bool = False,
                     info: dict | None = None):
    """Residual join of a block's output y [N, H] with the stream h [N, H]:

        u = norm(y) * w_post + b_post          (with a post-norm; else y)
        h_out = alpha * h + beta * act(gate) * u
        z = norm(h_out) * w_pre + b_pre        (with a pre-norm)

    Returns (h_out, z, stats); z is None without a pre-norm.  y and z are bf16 or fp32; the
    stream has that type or is fp32 (``stream_dtype``, for a join without h).  A post-norm is
    taken where w_post or b_post is given, unless ``post_norm`` says otherwise.  gate: a scalar or [H],
    learned, or [N, 1] or [N, H] with a value per token.  out may be h itself and z may be
    y.  ``checkpoint``, of [N, H], receives z in 8 bits."""
    lib = _library()
    _check_y(y)
    shape = y.shape
    N, H = shape
    dev, dt = y.device, y.dtype
    st = h.dtype if h is not None else stream_dtype or dt
    head, ga, vecs, _ = _common(dt, shape, dev, st, w_post, b_post, w_pre, b_pre, gate, gate_act,
                                kind, alpha, beta, eps, post_norm, pre_norm)
    if out is None:
        out = torch.empty(shape, dtype=st, device=dev)
    if not pre_norm:
        z = None
    elif z is None:
        z = torch.empty(shape, dtype=dt, device=dev)
    if stats is None:
        stats = torch.empty((4, N), dtype=torch.float32, device=dev)
    ck = 0
    if checkpoint is not None:
        if not pre_norm or (checkpoint.N, checkpoint.H) != (N, H) \
                or checkpoint.data.device != dev:
            raise ValueError(f"checkpoint must be of z, {(N, H)} on {dev}")
        ck = checkpoint.data.data_ptr()
    a = _pack(*head, *_rows("y", y, shape, dt, dev), *_rows("h", h, shape, st, dev), *ga, *vecs,
              *_rows("out", out, shape, st, dev), _check_stats(stats, N, dev),
              *_rows("z", z, shape, dt, dev), ck, *_NO_BACKWARD)
    _call(lib.flce_resnorm_fwd, dev, dt, (a,), sync=sync, workspace=None, info=info)
    return out, z, stats


_NO_BACKWARD = (0,) * 14


class ResnormGrads(NamedTuple):
    """Gradients of a residual join; None where there is no such input."""
    dy: torch.Tensor
    dh: torch.Tensor | None
    dgate: torch.Tensor | None
    dw_post: torch.Tensor | None
    db_post: torch.Tensor | None
    dw_pre: torch.Tensor | None
    db_pre: torch.Tensor | None


def flce_resnorm_bwd(dz: torch.Tensor | None, dh_out: torch.Tensor | None,
                     y: torch.Tensor | None, h_out: torch.Tensor | None, stats: torch.Tensor, *,
                     w_pre: torch.Tensor | None = None, b_pre: torch.Tensor | None = None,
                     w_post: torch.Tensor | None = None, b_post: torch.Tensor | None = None,
                     gate: torch.Tensor | None = None, gate_act: str | None = None,
                     kind: str = "rms", alpha: float = 1.0, beta: float = 1.0,
                     eps: float = 1e-6, pre_norm: bool = True, post_norm: bool | None = None,
                     need_dh: bool = True, stream_dtype: torch.dtype | None = None,
                     dtype: torch.dtype | None = None,
                     dy: torch.Tensor | None = None, dh: torch.Tensor | None = None,
                     sync: bool = False, workspace: torch.Tensor | None = None,
                     info: dict | None = None) -> ResnormGrads:
    """Gradients of ``flce_resnorm_fwd`` at y, h_out and stats as it left them.  dz is the
    gradient of z (None without a pre-norm), dh_out what reaches h_out besides (None:
    nothing).  dy may be dz itself and dh may be dh_out.  Gradients of weights, biases and
    learned gates are fp32; dy and per-token gates' have y's type, dh the stream's
    (``need_dh=False`` for a join without h).  y is read for a post-norm or a gate and may be
    None without them, h_out without a pre-norm; ``dtype`` is y's type then, where it is
    neither dz's nor dh_out's."""
    lib = _library()
    name, like = (("y", y) if y is not None else ("dz", dz) if dz is not None
                  else ("dh_out", dh_out))
    if like is None:
        raise ValueError("neither dz nor dh_out is given")
    _check_y(like, name)
    shape = like.shape
    N, H = shape
    dev, dt = like.device, dtype if dtype is not None and like is dh_out else like.dtype
    if dt not in _HALF:
        raise TypeError(f"unsupported dtype {dt} (bf16 or fp32)")
    st = (h_out.dtype if h_out is not None else dh_out.dtype if dh_out is not None
          else stream_dtype or dt)
    head, ga, vecs, gk = _common(dt, shape, dev, st, w_post, b_post, w_pre, b_pre, gate, gate_act,
                                 kind, alpha, beta, eps, post_norm, pre_norm)
    if (dz is not None) != bool(pre_norm):
        raise ValueError("dz goes with a pre-norm")
    if pre_norm and h_out is None:
        raise ValueError("a pre-norm's gradient needs h_out")
    if y is None and (gate is not None or head[3]):
        raise ValueError("gradients of a post-norm or a gate need y")
    if dy is None:
        dy = torch.empty(shape, dtype=dt, device=dev)
    if dh is None and need_dh:
        dh = torch.empty(shape, dtype=st, device=dev)
    dga = _NONE
    dgate = None
    if gk != GATE_NONE:
        dgate = torch.empty(gate.shape, dtype=dt if gk > GATE_CHANNEL else torch.float32,
                            device=dev)
        dga = dgate.data_ptr(), H if gk == GATE_FULL else 1
    one = (H,)  # (a tensor each: the views of a common one would take longer to make)
    d = [None if t is None else torch.empty(one, dtype=torch.float32, device=dev)
         for t in (w_post, b_post, w_pre, b_pre)]
    at = [0 if t is None else t.data_ptr() for t in d]
    a = _pack(*head, *_rows("y", y, shape, dt, dev), 0, 0, *ga, *vecs,
              *_rows("h_out", h_out, shape, st, dev), _check_stats(stats, N, dev), 0, 0, 0,
              *_rows("dz", dz, shape, dt, dev), *_rows("dh_out", dh_out, shape, st, dev),
              *_rows("dy", dy, shape, dt, dev), *_rows("dh", dh, shape, st, dev), *dga, *at)
    _call(lib.flce_resnorm_bwd, dev, dt, (a,), sync=sync, workspace=workspace, info=info)
    return ResnormGrads(dy, dh, dgate, *d)


def flce_ckpt_save(x: torch.Tensor, *, out: Checkpoint | None = None, sync: bool = False,
                   info: dict | None = None) -> Checkpoint:
    """x [N, H] (bf16 or fp32, contiguous last axis) in 8 bits."""
    lib = _library()
    _check_y(x, "x")
    N, H = x.shape
    if out is None:
        out = Checkpoint.empty(N, H, x.device)
    elif (out.N, out.H) != (N, H) or out.data.device != x.device:
        raise ValueError(f"out must be a checkpoint of {(N, H)} on {x.device}")
    _call(lib.flce_ckpt_save, x.device, x.dtype,
          (*_rows("x", x, x.shape, x.dtype, x.device), N, H, out.data.data_ptr()), sync=sync,
          workspace=None, info=info)
    return out


def flce_ckpt_load(ckpt: Checkpoint, *, dtype: torch.dtype = torch.bfloat16,
                   out: torch.Tensor | None = None, sync: bool = False,
                   info: dict | None = None) -> torch.Tensor:
    """The values that a checkpoint stands for, in bf16 (exactly) or fp32."""
    lib = _library()
    N, H, dev = ckpt.N, ckpt.H, ckpt.data.device
    if out is None:
        if dtype not in _HALF:
            raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
        out = torch.empty((N, H), dtype=dtype, device=dev)
    _dtype_code(out)
    p, row = _rows("out", out, (N, H), out.dtype, dev)
    _call(lib.flce_ckpt_load, dev, out.dtype, (ckpt.data.data_ptr(), N, H, p, row), sync=sync,
          workspace=None, info=info)
    return out


def flce_ckpt_wgrad(dY: torch.Tensor, ckpt: Checkpoint, *, dW: torch.Tensor | None = None,
                    accumulate: bool = False, sync: bool = False,
                    workspace: torch.Tensor | None = None,
                    info: dict | None = None) -> torch.Tensor:
    """``dW = dY^T X`` in fp32 [O, I] for dY [N, O] (bf16) and X [N, I] as ``ckpt`` holds it:
    the weight gradient of ``Y = X W^T``.  ``accumulate=True`` adds it to ``dW``."""
    lib = _library()
    _check_y(dY, "dY")
    if dY.dtype is not torch.bfloat16:
        raise TypeError(f"dY must be bf16, got {dY.dtype}")
    N, O = dY.shape
    I, dev = ckpt.H, dY.device
    if ckpt.N != N or ckpt.data.device != dev:
        raise ValueError(f"dY has {N} rows on {dev}, the checkpoint {ckpt.N} on "
                         f"{ckpt.data.device}")
    if dW is None:
        if accumulate:
            raise ValueError("give dW to accumulate into")
        dW = torch.empty((O, I), dtype=torch.float32, device=dev)
    else:
        _check_out(dW, (O, I), torch.float32, dev, "dW")
    _call(lib.flce_ckpt_wgrad, dev, dY.dtype,
          (*_rows("dY", dY, dY.shape, dY.dtype, dev), ckpt.data.data_ptr(), N, O, I,
           dW.data_ptr(), 1 if accumulate else 0), sync=sync, workspace=workspace, info=info)
    return dW


def _aligned(t):
    """t, or a copy of it that is contiguous and begins on 16 bytes."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _row_strided(t):
    """t itself if the library takes its strides and address, else a copy that it takes."""
    ok = (t.stride(1) == 1 and t.stride(0) >= t.shape[1] and t.stride(0) % 8 == 0
          and t.data_ptr() % 16 == 0)
    return t if ok else _aligned(t)


def _flat(t):
    """[..., n] as rows of n."""
    return t.reshape(math.prod(t.shape[:-1]), t.shape[-1])


def _as(grad, like):
    """A parameter's fp32 gradient in the parameter's type."""
    if grad is None or grad.dtype is like.dtype:
        return grad
    return scale_convert(grad, torch.empty(grad.shape, dtype=like.dtype, device=grad.device))


class _ResidualNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, h, w_pre, b_pre, w_post, b_post, gate, opts):
        y = _row_strided(y)
        h = None if h is None else _row_strided(h)
        params = [None if t is None else _aligned(t) for t in (w_pre, b_pre, w_post, b_post)]
        if gate is not None and gate.dim() == 2 and gate.shape[1] > 1:
            gate = _row_strided(gate)
        elif gate is not None:
            gate = _aligned(gate) if gate.dim() == 1 else gate.contiguous()
        kw = dict(zip(("w_pre", "b_pre", "w_post", "b_post"), params), gate=gate,
                  **{k: v for k, v in opts.items() if k != "checkpoint"})
        ck = Checkpoint.empty(*y.shape, y.device) if opts["checkpoint"] else None
        h_out, z, stats = flce_resnorm_fwd(y, h, checkpoint=ck, **kw)
        # what the gradients read: a plain pre-norm join keeps its stream and not y
        reads_y = gate is not None or params[2] is not None or params[3] is not None \
            or opts["post_norm"]
        ctx.save_for_backward(y if reads_y else None, h_out if opts["pre_norm"] else None, stats,
                              *params, gate)
        ctx.opts, ctx.has_h, ctx.dtype = opts, h is not None, y.dtype
        ctx.set_materialize_grads(False)
        if ck is None:
            return h_out, z, None
        ctx.mark_non_differentiable(ck.data)
        return h_out, z, ck.data

    @staticmethod
    @once_differentiable  # the kernels' results carry no graph of their own
    def backward(ctx, dh_out, dz, _):
        y, h_out, stats, w_pre, b_pre, w_post, b_post, gate = ctx.saved_tensors
        if dh_out is None and dz is None:
            return (None,) * 8
        # without a use of z its norm has no part in the gradients, whatever the stream holds
        opts = {k: v for k, v in ctx.opts.items() if k != "checkpoint"}
        unused = dz is None and opts["pre_norm"]
        g = flce_resnorm_bwd(
            None if dz is None else _row_strided(dz),
            None if dh_out is None else _row_strided(dh_out), y, None if unused else h_out, stats,
            w_pre=None if unused else w_pre, b_pre=None if unused else b_pre, w_post=w_post,
            b_post=b_post, gate=gate, need_dh=ctx.has_h, dtype=ctx.dtype,
            **{**opts, "pre_norm": dz is not None})
        dw_pre, db_pre = (_as(d, t) if d is not None or t is None else torch.zeros_like(t)
                          for d, t in ((g.dw_pre, w_pre), (g.db_pre, b_pre)))
        return (g.dy, g.dh, dw_pre, db_pre, _as(g.dw_post, w_post), _as(g.db_post, b_post),
                _as(g.dgate, gate), None)


class ResidualNorm(torch.nn.Module):
    """``join(y, h, w_pre=..., w_post=..., gate=...)`` -> (h_out, z): the residual stream and the
    next block's input, differentiable in every tensor.  With ``checkpoint=True`` it returns
    (h_out, z, checkpoint of z), for ``CheckpointedLinear``.  Leave ``h`` out for the
    first norm of a model: ``join(x, w_pre=w)``."""

    def __init__(self, kind: str = "rms", *, alpha: float = 1.0, beta: float = 1.0,
                 eps: float = 1e-6, gate_act: str | None = None, pre_norm: bool = True,
                 post_norm: bool | None = None, checkpoint: bool = False):
        super().__init__()
        if checkpoint and not pre_norm:
            raise ValueError("a checkpoint of z needs pre_norm")
        self.opts = dict(kind=kind, alpha=alpha, beta=beta, eps=eps, gate_act=gate_act,
                         pre_norm=pre_norm, post_norm=post_norm, checkpoint=checkpoint)

    def forward(self, y, h=None, *, w_pre=None, b_pre=None, w_post=None, b_post=None, gate=None):
        h_out, z, ck = _ResidualNormFunction.apply(y, h, w_pre, b_pre, w_post, b_post, gate,
                                                   self.opts)
        if ck is None:
            return h_out, z
        return h_out, z, Checkpoint(ck, *y.shape)


class _CheckpointedLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, saved, keep):
        flat = _row_strided(_flat(x))
        if saved is not None and (saved.N, saved.H) != tuple(flat.shape):
            raise ValueError(f"saved must be a checkpoint of {tuple(flat.shape)}")
        if keep and saved is None:
            saved = flce_ckpt_save(flat)
        ctx.save_for_backward(weight, saved.data if keep else None)
        ctx.shape = x.shape
        return (flat @ weight.t()).view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        weight, data = ctx.saved_tensors
        flat = _row_strided(_flat(grad_out))
        dx = dW = None
        if ctx.needs_input_grad[0]:
            dx = (flat @ weight).view(ctx.shape)
        if ctx.needs_input_grad[1]:
            ck = Checkpoint(data, flat.shape[0], weight.shape[1])
            dW = _as(flce_ckpt_wgrad(flat, ck), weight)
        return dx, dW, None, None


class CheckpointedLinear(torch.nn.Module):
    """``linear(x, weight, saved=None)`` -> ``x @ weight.T`` in bf16, whose backward pass takes
    the weight's gradient from x in 8 bits instead of x itself.  x [..., I], weight [O, I], O
    and I multiples of 8; ``saved`` is a checkpoint of x that another call made
    (``ResidualNorm``, or a linear that shares the input).  Where weight has no gradient to come
    (frozen, or under ``no_grad``) no checkpoint is made or kept."""

    def forward(self, x, weight, saved: Checkpoint | None = None):
        if x.dtype is not torch.bfloat16 or weight.dtype is not torch.bfloat16:
            raise TypeError("CheckpointedLinear takes bf16 x and weight")
        if weight.dim() != 2 or x.shape[-1:] != weight.shape[1:] \
                or weight.shape[0] % 8 or weight.shape[1] % 8:
            raise ValueError("x must be [..., I] and weight [O, I], O and I multiples of 8")
        if not x.is_cuda or weight.device != x.device \
                or (saved is not None and saved.data.device != x.device):
            raise ValueError("x, weight and saved must be on one CUDA device")
        keep = weight.requires_grad and torch.is_grad_enabled()
        if keep and not all(8 <= n <= 1 << 20 for n in weight.shape):
            raise ValueError("O and I of a weight with a gradient must be 8 .. 2^20")
        return _CheckpointedLinearFunction.apply(x, weight, saved, keep)
