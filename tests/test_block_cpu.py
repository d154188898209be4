"""CPU-only checks of the operators between blocks: the tests' plain forms against autograd
and differences, and what the C entries and the binding refuse before any device is touched."""
import ctypes

import pytest
import torch

import linear_cross_entropy_fwd_gb300 as flce
from block_util import dequantise, e4m3_table, join, join_grads, pre, quantise
from linear_cross_entropy_fwd_gb300 import build as flce_build

A = 1 << 20  # a non-null, aligned address; refused calls never read it
M = 1 << 30


@pytest.fixture(scope="module")
def lib():
    flce_build.build()
    return flce.load_library()


# ------------------------------------------------------------- the plain forms
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate,act", [(None, None), ((), "tanh"), ((16,), None),
                                      ((5, 1), "sigmoid"), ((5, 16), "tanh")])
@pytest.mark.parametrize("post_norm,pre_norm", [(True, True), (False, True), (True, False)])
def test_gradient_formulas(kind, gate, act, post_norm, pre_norm):
    """The formulas against autograd, and autograd against differences of the join."""
    g = torch.Generator().manual_seed(3)

    def t(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64)

    y, h, dz, dh = t(5, 16), t(5, 16), t(5, 16), t(5, 16)
    p = dict(w_pre=t(16) if pre_norm else None, b_pre=t(16) if pre_norm else None,
             w_post=t(16) if post_norm else None, b_post=t(16) if post_norm else None,
             gate=None if gate is None else t(*gate))
    opts = dict(kind=kind, gate_act=act, alpha=1.3, beta=0.6, eps=1e-3, post_norm=post_norm,
                pre_norm=pre_norm)
    leaves = {"dy": y, "dh": h, **{"d" + k: v for k, v in p.items() if v is not None}}
    for v in leaves.values():
        v.requires_grad_()

    def f(*_):
        out, _ = join(y, h, p, opts)
        s = (out * dh).sum()
        return s + (pre(out, p, opts)[0] * dz).sum() if pre_norm else s

    assert torch.autograd.gradcheck(f, tuple(leaves.values()))
    grads = dict(zip(leaves, torch.autograd.grad(f(), tuple(leaves.values()))))
    with torch.no_grad():
        h_out, _ = join(y, h, p, opts)
    got = join_grads(dz if pre_norm else None, dh, y.detach(), h_out,
                     {k: None if v is None else v.detach() for k, v in p.items()}, opts)
    for k, v in grads.items():
        assert torch.allclose(got[k][0], v, rtol=1e-10, atol=1e-10), k


def test_quantiser_definition():
    """Every e4m3 number at every kind of scale comes back as it is, the nearest is taken
    elsewhere, and ties go to even codes."""
    table = e4m3_table()[:127]
    assert table[126] == 448 and table[1] == 2.0 ** -9
    for e in (-117, -3, 0, 7, 8, 119):
        x = torch.zeros(4, 64, dtype=torch.float64)
        x.view(-1)[:127] = table * 2.0 ** e
        x[:, 31] = x[:, 63] = 448 * 2.0 ** e  # the scale of each group
        codes, scales = quantise(x)
        assert bool((scales[:, :2] == e + 127).all()) and not scales[:, 2:].any()
        assert torch.equal(dequantise(codes, scales, 64), x)
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, :6] = torch.tensor([448., 17., 19., -25., 2.0 ** -10, 3 * 2.0 ** -10])
    back = dequantise(*quantise(x), 32)[0, :6]
    assert back.tolist() == [448., 16., 20., -24., 0., 2.0 ** -8]
    x = torch.randn(7, 1000, generator=torch.Generator().manual_seed(1)).double()
    codes, scales = quantise(x)
    assert codes.shape == (7, 1024) and scales.shape == (7, 32) and not codes[:, 1000:].any()
    err = (dequantise(codes, scales, 1000) - x).abs()
    floor = 2.0 ** (scales[:, :32].double() - 127 - 10)
    tol = torch.maximum(x.abs() / 16, floor.repeat_interleave(32, 1)[:, :1000])
    assert bool((err <= tol).all())


# ------------------------------------------------------------------ refusals
def _join(**kw):
    """A flce_resnorm that no check refuses, with some fields replaced."""
    a = flce.FlceResnorm()
    f = dict(N=300, H=64, norm=0, post_norm=1, pre_norm=1, gate_kind=4, gate_act=1, alpha=1.0,
             beta=1.0, eps=1e-6, stats=A, w_post=A, b_post=A + 4096, w_pre=A + 8192,
             b_pre=A + 12288)
    f["stats"] = A + M
    for i, n in enumerate(("y", "h", "gate", "h_out", "z", "dz", "dh_out", "dy", "dh", "dgate")):
        f.update({n: A + (2 + i) * M, n + "_row": 64})
    for i, n in enumerate(("dw_post", "db_post", "dw_pre", "db_pre")):
        f[n] = A + (20 + i) * M
    f.update(kw)
    for n, x in f.items():
        setattr(a, n, x)
    return a


def _opts(dtype=flce.FLCE_BF16):
    """A workspace of 0 bytes keeps an accepted call off the GPU."""
    o = flce.make_opts(sync=1)
    o.dtype = dtype
    o.workspace, o.workspace_bytes = 256, 0
    return ctypes.byref(o)


ACCEPTED = (flce.FLCE_ERR_ARCH, flce.FLCE_ERR_CUDA, flce.FLCE_ERR_WORKSPACE)
ARG, ALIGN = flce.FLCE_ERR_ARG, flce.FLCE_ERR_ALIGN


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), ARG), (dict(N=1 << 31), ARG), (dict(H=0), ARG), (dict(H=12), ARG),
    (dict(H=16392), ARG), (dict(norm=2), ARG), (dict(norm=-1), ARG), (dict(gate_kind=5), ARG),
    (dict(gate_act=3), ARG), (dict(alpha=float("nan")), ARG), (dict(beta=float("inf")), ARG),
    (dict(eps=-1e-9), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(gate=None), ARG), (dict(gate_row=56), ARG), (dict(gate_row=68), ALIGN),
    (dict(gate_kind=1, gate=A + 3), ALIGN), (dict(gate_kind=2, gate=A + 8), ALIGN),
    (dict(gate_kind=3, gate_row=0), ARG), (dict(gate_kind=3, gate=A + 1), ALIGN),
    (dict(w_pre=A + 4), ALIGN), (dict(b_post=A + 2), ALIGN), (dict(y=None), ARG),
    (dict(y_row=56), ARG), (dict(y_row=-64), ARG), (dict(y_row=68), ALIGN),
    (dict(y=A + 2 * M + 8), ALIGN), (dict(y_row=1 << 38), ARG), (dict(h_out=None), ARG),
])
def test_resnorm_refusals_of_both(lib, kw, status):
    fwd = lib.flce_resnorm_fwd(ctypes.byref(_join(**kw)), _opts())
    if kw == dict(h_out=None):
        assert fwd in ACCEPTED  # the forward pass need not store the stream
    else:
        assert fwd == status and lib.flce_last_error()
    assert lib.flce_resnorm_bwd(ctypes.byref(_join(**kw)), _opts()) == status
    assert lib.flce_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), ARG), (dict(h_row=8), ARG), (dict(h=A + 8), ALIGN),
    (dict(pre_norm=0, h_out=None), ARG), (dict(pre_norm=0, z_ckpt=A + 40 * M), ARG),
    (dict(z_ckpt=A + 8), ALIGN), (dict(stats=A + M + 2), ALIGN),
])
def test_resnorm_forward_refusals(lib, kw, status):
    assert lib.flce_resnorm_fwd(ctypes.byref(_join(**kw)), _opts()) == status
    assert lib.flce_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dz=None), ARG), (dict(dy=None), ARG), (dict(stats=None), ARG),
    (dict(pre_norm=0, dh_out=None), ARG), (dict(dgate=None), ARG), (dict(dgate_row=8), ARG),
    (dict(gate_kind=2, dgate=None), ARG), (dict(gate_kind=1, dgate=A + 2), ALIGN),
    (dict(dh_row=72 + 4), ALIGN), (dict(dw_pre=A + 4), ALIGN),
])
def test_resnorm_backward_refusals(lib, kw, status):
    assert lib.flce_resnorm_bwd(ctypes.byref(_join(**kw)), _opts()) == status
    assert lib.flce_last_error()


def test_resnorm_accepts(lib):
    row = 64 * 2
    for kw in (dict(), dict(h=None, h_row=0), dict(stats=A + M), dict(stream_fp32=1),
               dict(params_fp32=1), dict(gate_kind=0, gate=None, dgate=None), dict(N=0),
               dict(h=A + 5 * M), dict(z=A + 2 * M), dict(dh=A + 8 * M), dict(dy=A + 7 * M),
               dict(N=1, y_row=0, h_row=0, z_row=-5), dict(z_ckpt=A + 40 * M),
               # y, h and z beside each other in one buffer
               dict(y=A + 50 * M, h=A + 50 * M + row, z=A + 50 * M + 2 * row, y_row=192,
                    h_row=192, z_row=192)):
        for fn in (lib.flce_resnorm_fwd, lib.flce_resnorm_bwd):
            assert fn(ctypes.byref(_join(**kw)), _opts()) in ACCEPTED, (kw, lib.flce_last_error())


@pytest.mark.parametrize("kw,forward", [
    (dict(h_out=A + 2 * M), True),                       # the stream over y
    (dict(z=A + 3 * M), True),                           # z over h
    (dict(z=A + 2 * M, z_row=128), True),                # z over y with another stride
    (dict(z=A + 2 * M + 128 * 299), True),               # into y's last row
    (dict(h_out=A + 3 * M + 128), True),                 # the stream one row off in place
    (dict(z=A + 4 * M), True),                           # z over the gate
    (dict(z=A + 5 * M), True),                           # z over h_out
    (dict(z=A), True),                                   # over a weight
    (dict(z_ckpt=A + 2 * M + 128), True),
    (dict(stats=A + 6 * M), True),
    (dict(y=A + 50 * M, z=A + 50 * M + 96, y_row=192, z_row=192), True),  # a part of each row
    (dict(dy=A + 2 * M), False),                         # dy over y
    (dict(dy=A + 5 * M), False),                         # dy over h_out
    (dict(dh=A + 7 * M), False),                         # dh over dz
    (dict(dh=A + 9 * M), False),                         # dh over dy
    (dict(dgate=A + 4 * M), False),
    (dict(dw_pre=A + 20 * M + 128), False),              # over dw_post
    (dict(dw_pre=A + 8192 + 64), False),                 # over a weight
    (dict(dh=A + 8 * M, dh_row=72), False),              # in place with another stride
])
def test_resnorm_refuses_overlaps(lib, kw, forward):
    fn = lib.flce_resnorm_fwd if forward else lib.flce_resnorm_bwd
    assert fn(ctypes.byref(_join(**kw)), _opts()) == ARG
    assert b"overlaps" in lib.flce_last_error()


def test_resnorm_other_refusals(lib):
    assert lib.flce_resnorm_fwd(None, _opts()) == ARG
    assert lib.flce_resnorm_bwd(ctypes.byref(_join()), _opts(7)) == ARG
    # in place with another type: an fp32 stream and bf16 y do not share rows
    assert lib.flce_resnorm_fwd(ctypes.byref(_join(stream_fp32=1, h=A + 5 * M, h_row=72)),
                                _opts()) == ARG


def test_checkpoint_bytes(lib):
    assert lib.flce_ckpt_bytes(3, 8) == 3 * (32 + 4)
    assert lib.flce_ckpt_bytes(3, 136) == 3 * (160 + 8)
    assert lib.flce_ckpt_bytes(65536, 4096) == 65536 * (4096 + 128)
    assert flce.checkpoint_bytes(0, 8) == 0
    for a in ((-1, 8), (1 << 31, 8), (1, 0), (1, (1 << 20) + 8)):
        assert lib.flce_ckpt_bytes(*a) == 0
        with pytest.raises(ValueError):
            flce.checkpoint_bytes(*a)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), ARG), (dict(N=1 << 31), ARG), (dict(H=0), ARG), (dict(H=(1 << 20) + 8), ARG),
    (dict(H=12), ALIGN), (dict(x=None), ARG), (dict(c=None), ARG), (dict(row=56), ARG),
    (dict(row=68), ALIGN), (dict(x=A + 8), ALIGN), (dict(c=A + M + 4), ALIGN),
    (dict(c=A + 128), ARG), (dict(x=A + M + 128), ARG), (dict(dtype=5), ARG),
    (dict(N=1 << 30, H=1 << 20, row=1 << 20), ARG),
])
def test_checkpoint_refusals(lib, kw, status):
    a = dict(N=300, H=64, x=A, row=64, c=A + M, dtype=flce.FLCE_BF16)
    a.update(kw)
    o = _opts(a["dtype"])
    assert lib.flce_ckpt_save(a["x"], a["row"], a["N"], a["H"], a["c"], o) == status
    assert lib.flce_last_error()
    assert lib.flce_ckpt_load(a["c"], a["N"], a["H"], a["x"], a["row"], o) == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), ARG), (dict(N=1 << 31), ARG), (dict(O=0), ARG), (dict(I=0), ARG),
    (dict(O=(1 << 20) + 8), ARG), (dict(O=12), ALIGN), (dict(I=4), ALIGN), (dict(dY=None), ARG),
    (dict(c=None), ARG), (dict(dW=None), ARG), (dict(row=56), ARG), (dict(row=68), ALIGN),
    (dict(dY=A + 8), ALIGN), (dict(c=A + 8), ALIGN), (dict(dW=A + 4), ALIGN),
    (dict(dW=A + 64), ARG), (dict(dW=A + M + 64), ARG), (dict(dtype=flce.FLCE_FP32), ARG),
])
def test_wgrad_refusals(lib, kw, status):
    a = dict(N=300, O=64, I=32, dY=A, row=64, c=A + M, dW=A + 2 * M, dtype=flce.FLCE_BF16)
    a.update(kw)
    for acc in (0, 1):
        assert lib.flce_ckpt_wgrad(a["dY"], a["row"], a["c"], a["N"], a["O"], a["I"], a["dW"],
                                   acc, _opts(a["dtype"])) == status
        assert lib.flce_last_error()


def test_binding_refusals():
    x = torch.zeros(3, 8)
    for call in (lambda: flce.flce_resnorm_fwd(x), lambda: flce.flce_ckpt_save(x),
                 lambda: flce.flce_resnorm_bwd(x, None, x, x, torch.zeros(4, 3)),
                 lambda: flce.Checkpoint(torch.zeros(108, dtype=torch.uint8), 3, 8)):
        with pytest.raises(ValueError):  # not on a device
            call()
    with pytest.raises(ValueError):
        flce.ResidualNorm(pre_norm=False, checkpoint=True)
