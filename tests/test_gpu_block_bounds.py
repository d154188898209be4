"""Bounds of the operators between blocks: every buffer they write lies in the middle of a
larger one whose other bytes have to survive, outputs start as NaN and have to be written
whole, and rows lie beyond 2^31 elements from a buffer's start."""
import pytest
import torch

from test_gpu_step_guard_bands import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def _randn(*shape, dtype=BF):
    return torch.randn(shape, device=DEV).to(dtype)


@pytest.mark.parametrize("N,H", [(1, 8), (5, 72), (400, 264), (9, 1000), (3, 2056), (2, 4104),
                                 (1, 16384), (700, 4096)])
@pytest.mark.parametrize("dt,st", [(BF, BF), (BF, FP), (FP, FP)])
@pytest.mark.parametrize("gate", ["token", "full", "channel"])
def test_resnorm_bounds(cuda_lib, N, H, dt, st, gate):
    flce = cuda_lib
    shape = {"token": (N, 1), "full": (N, H), "channel": (H,)}[gate]
    kw = dict(w_pre=_randn(H, dtype=dt), b_pre=_randn(H, dtype=dt), w_post=_randn(H, dtype=dt),
              b_post=_randn(H, dtype=dt), gate=_randn(*shape, dtype=dt), kind="layer")
    y, dz = _randn(N, H, dtype=dt), _randn(N, H, dtype=dt)
    h, dh_out = _randn(N, H, dtype=st), _randn(N, H, dtype=st)
    out = {"out": Guarded((N, H), st), "z": Guarded((N, H), dt), "stats": Guarded((4, N), FP)}
    ck = flce.Checkpoint.empty(N, H, DEV)
    data = Guarded((ck.data.numel(),), torch.uint8)
    ck.data = data.t
    flce.flce_resnorm_fwd(y, h, **kw, **{k: g.t for k, g in out.items()}, checkpoint=ck,
                          sync=True)
    data.check("checkpoint")
    args = (dz, dh_out, y, out["out"].t, out["stats"].t)
    info = {}
    flce.flce_resnorm_bwd(*args, **kw, info=info)
    ws = Guarded((info["workspace_bytes"],), torch.uint8)
    out.update(dy=Guarded((N, H), dt), dh=Guarded((N, H), st))
    flce.flce_resnorm_bwd(*args, **kw, dy=out["dy"].t, dh=out["dh"].t, workspace=ws.t, sync=True)
    ws.check("workspace")
    for name, g in out.items():
        g.check(name)


@pytest.mark.parametrize("N,H", [(1, 8), (3, 40), (70, 136), (33, 1000), (5, 4096)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_checkpoint_bounds(cuda_lib, N, H, dtype):
    x = _randn(N, H, dtype=dtype)
    data = Guarded((cuda_lib.checkpoint_bytes(N, H),), torch.uint8)
    ck = cuda_lib.Checkpoint(data.t, N, H)
    cuda_lib.flce_ckpt_save(x, out=ck, sync=True)
    data.check("checkpoint")
    back = Guarded((N, H), dtype)
    cuda_lib.flce_ckpt_load(ck, out=back.t, sync=True)
    back.check("x")
    data.check("checkpoint")


@pytest.mark.parametrize("N,O,I", [(1, 8, 8), (130, 264, 136), (64, 256, 512), (1000, 72, 1000),
                                   (9000, 520, 1032)])
def test_wgrad_bounds(cuda_lib, N, O, I):
    dY, ck = _randn(N, O), cuda_lib.flce_ckpt_save(_randn(N, I))
    dW = Guarded((O, I), FP)
    info = {}
    cuda_lib.flce_ckpt_wgrad(dY, ck, info=info)
    ws = Guarded((info["workspace_bytes"],), torch.uint8)
    for accumulate in (False, True):
        cuda_lib.flce_ckpt_wgrad(dY, ck, dW=dW.t, accumulate=accumulate, workspace=ws.t, sync=True)
        dW.check("dW")
        ws.check("workspace")


def test_far_rows(cuda_lib):
    """Row strides that put the last rows beyond 2^31 elements."""
    flce, N, H, stride = cuda_lib, 300, 264, 8_000_000
    rows = torch.empty(N * stride, dtype=BF, device=DEV).view(N, stride)
    names = ("y", "h", "gate", "dz", "dh_out", "out", "z", "dy", "dh", "x", "back")
    t = {n: rows[:, 1024 * i:1024 * i + H] for i, n in enumerate(names)}
    for n in ("y", "h", "gate", "dz", "dh_out", "x"):
        t[n].copy_(_randn(N, H))
    near = {n: v.contiguous() for n, v in t.items()}
    w = _randn(H)
    for kw in (dict(gate="gate"), dict()):
        far = dict(w_pre=w, w_post=w, gate=t["gate"] if kw else None)
        close = dict(w_pre=w, w_post=w, gate=near["gate"] if kw else None)
        a = flce.flce_resnorm_fwd(t["y"], t["h"], out=t["out"], z=t["z"], **far, sync=True)
        b = flce.flce_resnorm_fwd(near["y"], near["h"], **close)
        ga = flce.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], a[0], a[2], dy=t["dy"],
                                   dh=t["dh"], **far, sync=True)
        gb = flce.flce_resnorm_bwd(near["dz"], near["dh_out"], near["y"], b[0], b[2], **close)
        for u, v in zip(a + tuple(ga), b + tuple(gb)):
            assert (u is None and v is None) or torch.equal(u, v)
    ck = flce.flce_ckpt_save(t["x"], sync=True)
    assert torch.equal(ck.data, flce.flce_ckpt_save(near["x"]).data)
    assert torch.equal(flce.flce_ckpt_load(ck, out=t["back"], sync=True), flce.flce_ckpt_load(ck))
    assert torch.equal(flce.flce_ckpt_wgrad(t["dz"], ck, sync=True),
                       flce.flce_ckpt_wgrad(near["dz"], ck))


def test_many_elements(cuda_lib):
    """Checkpoints and joins of more than 2^31 elements."""
    N, H = 530_000, 4096
    x = torch.empty(N, H, dtype=BF, device=DEV)
    at = torch.tensor([0, 7, 262_143, 262_144, 524_287, 524_288, N - 1], device=DEV)
    x.fill_(0.5)
    x[at] = _randn(len(at), H)
    ck = cuda_lib.flce_ckpt_save(x, sync=True)
    few = cuda_lib.flce_ckpt_load(cuda_lib.flce_ckpt_save(x[at]))
    back = cuda_lib.flce_ckpt_load(ck, sync=True)
    assert torch.equal(back[at], few) and bool((back[1000] == 0.5).all())
    w = _randn(H)
    out, z, stats = cuda_lib.flce_resnorm_fwd(x, back, w_pre=w, out=back, sync=True)
    o2, z2, s2 = cuda_lib.flce_resnorm_fwd(x[at], few, w_pre=w)
    assert torch.equal(out[at], o2) and torch.equal(z[at], z2) and torch.equal(stats[:, at], s2)
    g = cuda_lib.flce_resnorm_bwd(z, out, x, out, stats, w_pre=w, dy=z, sync=True)
    g2 = cuda_lib.flce_resnorm_bwd(z2, o2, x[at], o2, s2, w_pre=w)
    assert torch.equal(g.dy[at], g2.dy) and torch.equal(g.dh[at], g2.dh)
