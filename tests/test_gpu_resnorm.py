"""The residual join and its gradients against 64-bit forms; block_util has the tolerances:
half a step of the output's type, and the roundings of fp32 on the way there."""
import itertools

import pytest
import torch

import block_util as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def _make(N, H, dt, st, pt, post=False, bias=False, gate="none", act=None, kind="rms", alpha=1.0,
          beta=1.0, eps=1e-6, pre_norm=True, weights=True, h=True, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(seed + N + H)

    def r(*s, t, std=1.0, mean=0.0):
        return (mean + std * torch.randn(s, generator=g)).to(t).to(DEV)

    shape = {"none": None, "scalar": (), "channel": (H,), "token": (N, 1), "full": (N, H)}[gate]
    p = dict(w_pre=r(H, t=pt, mean=1.0) if pre_norm and weights else None,
             b_pre=r(H, t=pt) if pre_norm and bias else None,
             w_post=r(H, t=pt, mean=1.0) if post and weights else None,
             b_post=r(H, t=pt) if post and bias else None,
             gate=None if shape is None else r(*shape, t=pt if len(shape) < 2 else dt))
    opts = dict(kind=kind, gate_act=act, alpha=alpha, beta=beta, eps=eps, post_norm=post,
                pre_norm=pre_norm)
    t = dict(y=r(N, H, t=dt, mean=offset), h=r(N, H, t=st, std=3.0) if h else None,
             dz=r(N, H, t=dt) if pre_norm else None, dh_out=r(N, H, t=st))
    return t, p, opts


def _forward(flce, t, p, opts, **kw):
    st = None if t["dh_out"] is None else t["dh_out"].dtype
    return flce.flce_resnorm_fwd(t["y"], t["h"], **p, **opts, stream_dtype=st, **kw)


def _check_forward(t, p, opts, out, z):
    ref.check(out, *ref.join(t["y"], t["h"], p, opts), "h_out")
    if opts["pre_norm"]:
        ref.check(z, *ref.pre(out, p, opts), "z")


def _check_backward(t, p, opts, out, got):
    want = ref.join_grads(t["dz"], t["dh_out"], t["y"], out, p, opts)
    for k, v in got._asdict().items():
        if v is not None:
            assert v.shape == want[k][0].shape, k
            ref.check(v, *want[k], k)


def _both(flce, N, H, dt, st, pt, **kw):
    t, p, opts = _make(N, H, dt, st, pt, **kw)
    out, z, stats = _forward(flce, t, p, opts, sync=True)
    _check_forward(t, p, opts, out, z)
    got = flce.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts,
                                need_dh=t["h"] is not None, sync=True)
    _check_backward(t, p, opts, out, got)
    again = flce.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts,
                                  need_dh=t["h"] is not None)
    for a, b in zip(got, again):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    return t, p, opts, out, z, stats, got


# rows of one warp and of several, of a part of a warp, of more than a CTA's warps
SIZES = [(1, 8), (1, 4096), (3, 64), (33, 72), (5, 264), (300, 136), (77, 1000), (19, 2056),
         (170, 4096), (9, 4104), (40, 8192), (7, 8200), (90, 16384)]
TYPES = [(BF, BF, BF), (BF, BF, FP), (BF, FP, BF), (BF, FP, FP), (FP, FP, FP)]


@pytest.mark.parametrize("N,H", SIZES)
@pytest.mark.parametrize("types", TYPES)
def test_sizes_and_types(cuda_lib, N, H, types):
    _both(cuda_lib, N, H, *types)
    _both(cuda_lib, N, H, *types, kind="layer", post=True, bias=True, gate="full", act="sigmoid",
          alpha=0.5, beta=1.25)


@pytest.mark.parametrize("kind,post,bias,gate", list(itertools.product(
    ["rms", "layer"], [False, True], [False, True],
    ["none", "scalar", "channel", "token", "full"])))
def test_forms(cuda_lib, kind, post, bias, gate):
    acts = [None] if gate == "none" else [None, "sigmoid", "tanh"]
    for i, act in enumerate(acts):
        _both(cuda_lib, 45, 200, *TYPES[i], kind=kind, post=post, bias=bias, gate=gate, act=act,
              alpha=1.5, beta=0.25, seed=i)
    # rows that a cluster shares
    _both(cuda_lib, 5, 4200, BF, BF, FP, kind=kind, post=post, bias=bias, gate=gate,
          act=acts[-1])


@pytest.mark.parametrize("types", [TYPES[0], TYPES[3]])
@pytest.mark.parametrize("kw", [
    dict(h=False), dict(h=False, weights=False), dict(pre_norm=False),
    dict(pre_norm=False, post=True, gate="channel"), dict(weights=False, post=True),
    dict(weights=False, post=True, bias=True, kind="layer"), dict(eps=1.0), dict(beta=0.0),
    dict(alpha=-1.0, beta=-2.0, post=True, gate="token", act="tanh"),
    dict(h=False, pre_norm=False, post=True), dict(kind="layer", offset=30.0, post=True),
])
def test_parts_left_out(cuda_lib, types, kw):
    _both(cuda_lib, 61, 320, *types, **kw)


def test_many_rows(cuda_lib):
    """More rows than the grid takes at once, in every launch shape."""
    for N, H in ((20011, 64), (3001, 1000), (1003, 4096), (333, 8192), (157, 12296)):
        _both(cuda_lib, N, H, BF, BF, BF, post=True, gate="channel")


@pytest.mark.parametrize("gate", ["none", "scalar", "channel", "token", "full"])
@pytest.mark.parametrize("kind,post,bias", [("layer", True, True), ("rms", False, False)])
def test_many_rows_of_every_gate(cuda_lib, gate, kind, post, bias):
    """As above; what a row leaves for the next one's sums, and the sums of the groups."""
    act = "none" if gate == "none" else "sigmoid"
    for N, H in ((20011, 64), (3001, 1000), (1003, 4096), (333, 8192), (157, 12296)):
        _both(cuda_lib, N, H, BF, FP if H == 1000 else BF, FP, kind=kind, post=post, bias=bias,
              gate=gate, act=act)


@pytest.mark.parametrize("gate", ["token", "channel", "full"])
@pytest.mark.parametrize("kind,bias", [("rms", False), ("layer", True)])
def test_nan_among_many_rows(cuda_lib, gate, kind, bias):
    """Rows that come before and after one with NaN or infinities in the same warps."""
    for N, H in ((5000, 64), (2500, 1000), (500, 4096), (300, 8192)):
        t, p, opts = _make(N, H, BF, BF, BF, kind=kind, post=True, bias=bias, gate=gate,
                           act="tanh")
        out, z, stats = _forward(cuda_lib, t, p, opts)
        got = cuda_lib.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts)
        bad = torch.zeros(N, dtype=torch.bool, device=DEV)
        bad[::7] = True
        t["y"][::14, 11], t["h"][7::14, H - 1] = float("nan"), float("inf")
        if gate != "channel":
            p["gate"][::21, -1] = float("inf")  # of a bad row too; a tanh of 1
            bad[::21] = True
        out2, z2, stats2 = _forward(cuda_lib, t, p, opts)
        for a, b in ((out, out2), (z, z2)):
            assert torch.equal(a[~bad], b[~bad])
        t["dz"][3::91, 5], t["dh_out"][5::91, 7] = float("nan"), float("-inf")
        bad[3::91] = bad[5::91] = True
        got2 = cuda_lib.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out2, stats2, **p, **opts)
        names = ["dy", "dh"] + (["dgate"] if gate != "channel" else [])
        for n in names:
            a, b = getattr(got, n), getattr(got2, n)
            assert torch.equal(a[~bad], b[~bad]), (n, N, H)


@pytest.mark.parametrize("kw", [dict(), dict(gate="full", act="sigmoid"), dict(h=False),
                                dict(gate="token", bias=True, alpha=0.5)])
def test_rows_that_are_asked_for_late(cuda_lib, kw):
    """bf16 rows of RMS norms without one after the block, 40 or more to a group of warps."""
    for N, H in ((97301, 264), (6101, 8192)):
        t, p, opts = _make(N, H, BF, BF, BF, **kw)
        out, z, stats = _forward(cuda_lib, t, p, opts, sync=True)
        _check_forward(t, p, opts, out, z)
        few, zf, sf = cuda_lib.flce_resnorm_fwd(
            t["y"][:99], None if t["h"] is None else t["h"][:99],
            **{**p, "gate": None if p["gate"] is None else p["gate"][:99]}, **opts)
        assert torch.equal(few, out[:99]) and torch.equal(zf, z[:99])
        assert torch.equal(sf, stats[:, :99])
        z2 = t["y"].clone()
        h2 = None if t["h"] is None else t["h"].clone()
        cuda_lib.flce_resnorm_fwd(z2, h2, **p, **opts, out=h2, z=z2)
        assert torch.equal(z2, z) and (h2 is None or torch.equal(h2, out))


def test_no_gradient_on_the_stream(cuda_lib):
    t, p, opts = _make(33, 128, BF, BF, BF, post=True, gate="scalar", act="tanh")
    out, _, stats = _forward(cuda_lib, t, p, opts)
    t["dh_out"] = None
    got = cuda_lib.flce_resnorm_bwd(t["dz"], None, t["y"], out, stats, **p, **opts)
    _check_backward(t, p, opts, out, got)


def test_gradients_wanted_in_part(cuda_lib):
    """Without weights their gradients are not computed; the others keep their bits."""
    t, p, opts = _make(33, 128, FP, FP, FP, kind="layer", post=True, bias=True)
    out, _, stats = _forward(cuda_lib, t, p, opts)
    full = cuda_lib.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts)
    none = cuda_lib.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts,
                                     need_dh=False)
    assert none.dh is None and torch.equal(none.dy, full.dy)


@pytest.mark.parametrize("H", [40, 1000, 4096, 5000])
def test_strides_and_in_place(cuda_lib, H):
    """Slices of one buffer, a stream updated in place, z over y, dy over dz, dh over dh_out."""
    flce, N = cuda_lib, 37
    t, p, opts = _make(N, H, BF, BF, BF, post=True, gate="full")
    out, z, stats = _forward(flce, t, p, opts)
    got = flce.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts)
    wide = torch.full((N, 6 * H + 16), 7.0, dtype=BF, device=DEV)
    names = ["y", "h", "dz", "dh_out"]
    s = {n: wide[:, i * H:(i + 1) * H] for i, n in enumerate(names)}
    for n in names:
        s[n].copy_(t[n])
    gate = wide[:, 4 * H:5 * H]
    gate.copy_(p["gate"])
    q = {**p, "gate": gate}
    o2, z2, st2 = flce.flce_resnorm_fwd(s["y"], s["h"], **q, **opts, out=s["h"],
                                        z=wide[:, 5 * H:6 * H])
    assert torch.equal(o2, out) and torch.equal(z2, z) and torch.equal(st2, stats)
    g2 = flce.flce_resnorm_bwd(s["dz"], s["dh_out"], s["y"], o2, st2, **q, **opts, dy=s["dz"],
                               dh=s["dh_out"])
    for a, b in zip(got, g2):
        assert (a is None and b is None) or torch.equal(a, b)
    assert bool((wide[:, 6 * H:] == 7).all())
    y = t["y"].clone()
    _, z3, _ = flce.flce_resnorm_fwd(y, t["h"], **p, **opts, z=y)
    assert torch.equal(y, z) and z3 is y


@pytest.mark.parametrize("N,H", [(3, 8), (21, 264), (9, 4104)])
@pytest.mark.parametrize("types", [TYPES[2], TYPES[4]])
def test_addresses_of_16_bytes(cuda_lib, N, H, types):
    """Rows that begin 16 bytes past a multiple of 32, and per-token gates that begin and end
    within a word, in tensors that end where the last of them does."""
    flce = cuda_lib
    t, p, opts = _make(N, H, *types, post=True, gate="token", act="tanh")
    out, z, stats = _forward(flce, t, p, opts)
    got = flce.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts)

    def off(x, like=None):
        n = 16 // x.element_size()
        raw = torch.empty(x.numel() + n, dtype=x.dtype, device=DEV)
        raw[n:] = x.reshape(-1)
        return raw[n:].view(x.shape)

    s = {k: off(v) for k, v in t.items()}
    raw = torch.empty(N + 1, dtype=p["gate"].dtype, device=DEV)
    raw[1:] = p["gate"][:, 0]
    q = {**p, "gate": raw[1:].view(N, 1)}
    o2, z2, st2 = flce.flce_resnorm_fwd(s["y"], s["h"], **q, **opts, out=off(out), z=off(z))
    assert torch.equal(o2, out) and torch.equal(z2, z) and torch.equal(st2, stats)
    g2 = flce.flce_resnorm_bwd(s["dz"], s["dh_out"], s["y"], o2, st2, **q, **opts,
                               dy=off(t["y"]), dh=off(t["h"]))
    for a, b in zip(got, g2):
        assert (a is None and b is None) or torch.equal(a, b)


def test_nan_and_infinity_stay_in_their_rows(cuda_lib):
    for kind, H in (("rms", 200), ("layer", 200), ("rms", 5000)):
        t, p, opts = _make(40, H, BF, BF, BF, kind=kind, post=True, gate="full", act="sigmoid")
        out, z, stats = _forward(cuda_lib, t, p, opts)
        got = cuda_lib.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts)
        bad = torch.zeros(40, dtype=torch.bool, device=DEV)
        for i, (n, v) in enumerate([("y", "nan"), ("h", "inf"), ("y", "-inf"), ("h", "nan")]):
            t[n][5 * i + 2, 11] = float(v)
            bad[5 * i + 2] = True
        p["gate"][30, 3], bad[30] = float("nan"), True
        out2, z2, stats2 = _forward(cuda_lib, t, p, opts)
        for a, b in ((out, out2), (z, z2)):
            assert torch.equal(a[~bad], b[~bad])
            assert bool((~torch.isfinite(b[bad])).any(1).all())
        t["dz"][33, 5], t["dh_out"][35, 7] = float("nan"), float("inf")
        bad[33] = bad[35] = True
        got2 = cuda_lib.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out2, stats2, **p, **opts)
        for a, b in ((got.dy, got2.dy), (got.dh, got2.dh), (got.dgate, got2.dgate)):
            assert torch.equal(a[~bad], b[~bad])
        assert bool(got2.dw_pre.isnan().any())


def test_extreme_values(cuda_lib):
    """A row of zeros with eps, the largest and smallest rows, and eps = 0."""
    N, H = 4, 512
    y = torch.randn(N, H, device=DEV)
    y[0] = 0
    y[1] *= 1e18
    y[2] *= 1e-18
    for kind in ("rms", "layer"):
        _, z, stats = cuda_lib.flce_resnorm_fwd(y, kind=kind, eps=1e-6)
        want, _, _, mag, _ = ref.norm(y.double(), kind, 1e-6, None, None)
        ref.check(z, want, ref.ROUNDS * ref.U * mag, kind)
        assert not z[0].any()
        big, small = 1e38 * torch.rand(1, H, device=DEV), 1e-38 * torch.randn(1, H, device=DEV)
        for x, eps in ((big, 1e-6), (big, 0.0), (small, 0.0), (small, 1e-38), (small, 1e-6)):
            _, z, _ = cuda_lib.flce_resnorm_fwd(x, kind=kind, eps=eps)
            # the kernel's eps is fp32's next number
            eps = torch.tensor(eps).double().item()
            want, _, _, mag, _ = ref.norm(x.double(), kind, eps, None, None)
            ref.check(z, want, ref.ROUNDS * ref.U * mag + 2.0 ** -140, kind)
        _, z, _ = cuda_lib.flce_resnorm_fwd(y[1:3], kind=kind, eps=0.0)
        want, _, _, mag, _ = ref.norm(y[1:3].double(), kind, 0.0, None, None)
        ref.check(z, want, ref.ROUNDS * ref.U * mag, kind)


def test_empty(cuda_lib):
    t, p, opts = _make(0, 64, BF, BF, FP, post=True, bias=True, gate="channel")
    out, z, stats = _forward(cuda_lib, t, p, opts, sync=True)
    assert out.shape == z.shape == (0, 64)
    got = cuda_lib.flce_resnorm_bwd(t["dz"], t["dh_out"], t["y"], out, stats, **p, **opts,
                                    sync=True)
    for n in ("dgate", "dw_post", "db_post", "dw_pre", "db_pre"):
        assert getattr(got, n).shape == (64,) and not getattr(got, n).any()
    y = torch.zeros(0, 64, dtype=BF, device=DEV, requires_grad=True)
    w = torch.ones(64, device=DEV, requires_grad=True)
    h, z = cuda_lib.ResidualNorm()(y, y, w_pre=w)
    (h.sum() + z.sum()).backward()  # gradients that are one number, spread over no rows
    assert y.grad.shape == (0, 64) and not w.grad.any()


def test_checkpoint_of_z(cuda_lib):
    """The checkpoint that the join leaves is that of the z it stores, bit for bit."""
    for (N, H), (dt, st, pt) in itertools.product(
            [(1, 8), (33, 72), (9, 1000), (50, 4096), (5, 8200)], [TYPES[0], TYPES[4]]):
        t, p, opts = _make(N, H, dt, st, pt, post=True, gate="channel")
        ck = cuda_lib.Checkpoint.empty(N, H, DEV)
        ck.data.fill_(0xA5)
        plain = _forward(cuda_lib, t, p, opts)
        with_ck = _forward(cuda_lib, t, p, opts, checkpoint=ck)
        assert all(torch.equal(a, b) for a, b in zip(plain, with_ck))
        assert torch.equal(ck.data, cuda_lib.flce_ckpt_save(with_ck[1]).data)


def test_other_stream_and_workspace(cuda_lib):
    """On another stream than the default, with the caller's workspace, two calls in flight."""
    t, p, opts = _make(500, 1024, BF, BF, BF, post=True, gate="channel")
    out, _, stats = _forward(cuda_lib, t, p, opts)
    args = (t["dz"], t["dh_out"], t["y"], out, stats)
    info = {}
    want = cuda_lib.flce_resnorm_bwd(*args, **p, **opts, info=info)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            ws = torch.empty(info["workspace_bytes"], dtype=torch.uint8, device=DEV)
            got.append(cuda_lib.flce_resnorm_bwd(*args, **p, **opts, workspace=ws))
    torch.cuda.synchronize()
    for g in got:
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(want, g))
    with pytest.raises(cuda_lib.FlceError) as e:
        cuda_lib.flce_resnorm_bwd(*args, **p, **opts,
                                  workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == cuda_lib.FLCE_ERR_WORKSPACE


def test_binding_refusals(cuda_lib):
    y, w = torch.zeros(3, 64, dtype=BF, device=DEV), torch.zeros(64, device=DEV)
    f = cuda_lib.flce_resnorm_fwd
    for err, call in [
            (TypeError, lambda: f(y.half())), (ValueError, lambda: f(y[0])),
            (ValueError, lambda: f(y.t())), (ValueError, lambda: f(y, y[:2])),
            (TypeError, lambda: f(y, y.half())), (TypeError, lambda: f(y.float(), y)),
            (ValueError, lambda: f(y, w_pre=w[:32])), (TypeError, lambda: f(y, w_pre=w.half())),
            (TypeError, lambda: f(y, w_pre=w, b_pre=w.to(BF))),
            (TypeError, lambda: f(y, gate=w, w_pre=w.to(BF))),
            (ValueError, lambda: f(y, gate=y[:2])), (ValueError, lambda: f(y, gate=w[:3])),
            (TypeError, lambda: f(y, gate=torch.zeros(3, 1, device=DEV))),
            (ValueError, lambda: f(y, kind="batch")), (ValueError, lambda: f(y, gate_act="relu")),
            (ValueError, lambda: f(y, w_post=w, post_norm=False)),
            (ValueError, lambda: f(y, w_pre=w, pre_norm=False)),
            (ValueError, lambda: f(y, out=torch.zeros(3, 72, dtype=BF, device=DEV))),
            (ValueError, lambda: f(y, checkpoint=cuda_lib.Checkpoint.empty(2, 64, DEV))),
            (cuda_lib.FlceError, lambda: f(y[:, :12])), (cuda_lib.FlceError, lambda: f(y, out=y)),
            (ValueError, lambda: cuda_lib.flce_resnorm_bwd(None, y, y, y, w))]:
        with pytest.raises(err):
            call()
