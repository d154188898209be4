"""Edges of the operators between blocks: arguments that a form does not use, sums
over tokens that are exact."""
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


# --------------------------------------------------------------- sums over tokens
@pytest.mark.parametrize("gate", ["none", "scalar", "channel", "token", "full"])
@pytest.mark.parametrize("kind,bias", [("rms", False), ("rms", True), ("layer", True)])
@pytest.mark.parametrize("post", [False, True])
def test_sums_over_tokens_are_exact(cuda_lib, gate, kind, bias, post):
    """Of small whole numbers, whose sums fp32 holds exactly in any order: a row that is left out,
    or counted twice, shows.  Statistics are an input of the gradients, and whole numbers too
    here.  Without a pre-norm dt is dh_out; with one its means are divided by H, and the
    sums that do not contain it are looked at."""
    for i, (N, H) in enumerate(((20011, 64), (3001, 1000), (1003, 4096), (333, 8192),
                                (157, 12296))):
        g = torch.Generator(device=DEV).manual_seed(i)

        def r(*shape, lo=0, hi=2, dtype=BF):
            return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).to(dtype)

        shape = {"none": None, "scalar": (), "channel": (H,), "token": (N, 1), "full": (N, H)}[gate]
        gt = None if shape is None else r(*shape, lo=1, dtype=FP if len(shape) < 2 else BF)
        layer = kind == "layer"
        stats = torch.ones(4, N, device=DEV)
        stats[0], stats[2] = (r(N, hi=1, dtype=FP), r(N, hi=1, dtype=FP)) if layer else (0, 0)
        y, h_out, dz, dh = r(N, H), r(N, H), r(N, H), r(N, H, lo=1)
        if H == 1000:
            h_out, dh = h_out.float(), dh.float()
        w_post, b_post = (r(H, lo=1, dtype=FP), r(H, hi=1, dtype=FP)) if post else (None, None)
        if not bias:
            b_post = None
        kw = dict(w_post=w_post, b_post=b_post, gate=gt, kind=kind, post_norm=post)
        yh = y.double() - (stats[0].double()[:, None] if post else 0)
        xh = h_out.double() - stats[2].double()[:, None]
        u = yh * w_post.double() if post else yh
        u = u if b_post is None else u + b_post.double()
        a = 1.0 if gt is None else gt.double()
        dt = dh.double()
        want = {}
        if post:
            want["dw_post"] = (yh * a * dt).sum(0)
            if bias:
                want["db_post"] = (a * dt).expand(N, H).sum(0)
        if gt is not None:
            dg = u * dt
            want["dgate"] = (dg.sum() if gate == "scalar" else dg.sum(0) if gate == "channel" else
                             dg.sum(1, keepdim=True).to(BF).double() if gate == "token" else dg)
        assert float((u * dt).abs().sum()) < 2 ** 24
        got = cuda_lib.flce_resnorm_bwd(None, dh, y, None, stats, **kw, pre_norm=False, sync=True)
        for k, v in want.items():
            assert torch.equal(getattr(got, k).double(), v), (k, N, H)
        kw.update(w_pre=r(H, lo=1, dtype=FP), b_pre=r(H, dtype=FP) if bias else None)
        got = cuda_lib.flce_resnorm_bwd(dz, dh, y, h_out, stats, **kw, sync=True)
        assert torch.equal(got.dw_pre.double(), (dz.double() * xh).sum(0)), (N, H)
        if bias:
            assert torch.equal(got.db_pre.double(), dz.double().sum(0)), (N, H)
