"""Edges of the operators between blocks: arguments that a form does not use."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def _randn(*shape, dtype=BF, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


# ------------------------------------------------- vectors of a norm that there is not
def _c_join(flce, fn, fields, dtype=BF):
    a = flce.FlceResnorm()
    a.alpha, a.beta, a.eps = 1.0, 1.0, 1e-6
    for n, v in fields.items():
        if torch.is_tensor(v):
            setattr(a, n, v.data_ptr())
            if hasattr(a, n + "_row"):
                setattr(a, n + "_row", v.stride(0) if v.dim() == 2 else 0)
        else:
            setattr(a, n, v)
    o = flce.make_opts(sync=1)
    o.dtype = flce.FLCE_BF16 if dtype is BF else flce.FLCE_FP32
    o.stream = torch.cuda.current_stream().cuda_stream
    assert fn(ctypes.byref(a), ctypes.byref(o)) == 0, flce.load_library().flce_last_error()


@pytest.mark.parametrize("N,H", [(3, 64), (300, 264), (6500, 4096), (5, 8200)])
@pytest.mark.parametrize("absent", ["post", "pre"])
@pytest.mark.parametrize("gate", [0, 2, 4])
def test_vectors_without_their_norm(cuda_lib, N, H, absent, gate):
    """u = y without a post-norm and there is no z without a pre-norm, whatever w_post, b_post,
    w_pre and b_pre of the structure point to; their gradients are not written."""
    flce, lib = cuda_lib, cuda_lib.load_library()
    w, b = _randn(H, seed=1), _randn(H, seed=2)
    t = dict(N=N, H=H, norm=1, post_norm=int(absent != "post"), pre_norm=int(absent != "pre"),
             gate_kind=gate, gate_act=1, y=_randn(N, H, seed=3), h=_randn(N, H, seed=4),
             dz=_randn(N, H, seed=5), dh_out=_randn(N, H, seed=6))
    if gate:
        t["gate"] = _randn(H) if gate == 2 else _randn(N, H, seed=7)
    other = "pre" if absent == "post" else "post"
    t["w_" + other] = _randn(H, seed=8)
    got = []
    for extra in ({}, {"w_" + absent: w, "b_" + absent: b}):
        out = dict(h_out=torch.full((N, H), 3.0, dtype=BF, device=DEV),
                   z=torch.full((N, H), 3.0, dtype=BF, device=DEV),
                   stats=torch.full((4, N), 3.0, device=DEV))
        _c_join(flce, lib.flce_resnorm_fwd, {**t, **extra, **out})
        g = dict(dy=torch.zeros(N, H, dtype=BF, device=DEV),
                 dh=torch.zeros(N, H, dtype=BF, device=DEV))
        if gate:
            g["dgate"] = torch.zeros(N, H, dtype=BF, device=DEV) if gate == 4 \
                else torch.zeros(H, device=DEV)
        g.update({"d" + k: torch.full((H,), 3.0, device=DEV)
                  for k in ("w_pre", "b_pre", "w_post", "b_post")})
        _c_join(flce, lib.flce_resnorm_bwd, {**t, **extra, **out, **g})
        got.append({**out, **g})
    for k, v in got[0].items():
        assert torch.equal(v, got[1][k]), k
    for k in ("dw_", "db_"):
        assert bool((got[1][k + absent] == 3).all())
    u = t["y"] if absent == "post" else None
    if u is not None and gate == 0:
        assert torch.equal(got[1]["h_out"], (t["h"].float() + u.float()).to(BF))
