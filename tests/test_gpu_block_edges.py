"""Edges of the operators between blocks: arguments that a form does not use, sums
over tokens that are exact, gates far from zero, and what the modules take and keep."""
import ctypes
import math
from types import SimpleNamespace

import pytest
import torch

import block_util as ref

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


# ------------------------------------------------------------------------- gates
UNITS = {"sigmoid": 3.5, "tanh": 2}


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("kind", ["full", "token", "channel", "scalar"])
def test_gates_far_from_zero(cuda_lib, act, kind):
    """act(gate) alone, as the join of ones: no h, beta 1, no norms.  The sigmoid is e or 1 over
    1 + e with e = exp(-|g|): the exponential is within 1 unit in the last place, 2^-23, the sum
    rounds once, the quotient is within 2 units: 3.5 2^-23 of the result, and 2 2^-149 where that is
    subnormal.  tanhf is within 2 units."""
    N, H = 16, 512
    far = torch.cat([torch.linspace(-110, 110, N * H // 2),
                     torch.logspace(-30, 0.5, N * H // 4), -torch.logspace(-30, 0.5, N * H // 4)])
    far[:3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    far = far.to(DEV)
    if kind == "full":
        gates = [far.view(N, H)]
    elif kind == "token":
        gates = [far[i::8].reshape(-1, 1) for i in range(8)]
    elif kind == "channel":
        gates = [far[i:i + H] for i in range(0, N * H, H)]
    else:
        gates = [far[i] for i in range(0, N * H, 301)]
    for g in gates:
        rows = g.shape[0] if kind in ("full", "token") else 2
        y = torch.ones(rows, H, device=DEV)
        got, _, _ = cuda_lib.flce_resnorm_fwd(y, gate=g, gate_act=act, pre_norm=False, sync=True)
        want = ref.ACT[act](g.double()).expand(rows, H)
        nan = want.isnan()
        assert torch.equal(got.isnan(), nan)
        err = (got.double() - want).abs()[~nan]
        tol = UNITS[act] * 2.0 ** -23 * want[~nan].abs() + 2.0 ** -148
        assert bool((err <= tol).all()), (float((err / tol).max()),
                                          float(g.expand(rows, H)[~nan][(err / tol).argmax()]))


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("kind", ["full", "token", "channel", "scalar"])
def test_gradients_of_gates_far_from_zero(cuda_lib, act, kind):
    """dy = act(gate) dt likewise; dgate's slope is a (1 - a) or 1 - a^2 of the activation in
    fp32, off by that activation's error, 4 2^-23 of 1 (a sigmoid's times 1 - 2 a, a tanh's 2
    units times 2 a), and three roundings of numbers up to 1; sums of up to 128 of them round about
    ten times more, 2^-24 of the sum each.  8 + 3 + 10 times 2^-24, below 2^-19."""
    N, H = 16, 64
    far = torch.linspace(-60, 60, N * H, device=DEV)
    shape = {"full": (N, H), "token": (N * H, 1), "channel": (16, H), "scalar": (1024,)}[kind]
    gates = [far.view(shape)] if kind in ("full", "token") else \
        list(far.view(shape)) if kind == "channel" else list(far[::37])
    for g in gates:
        rows = g.shape[0] if kind in ("full", "token") else 2
        y = torch.ones(rows, H, device=DEV)
        got = cuda_lib.flce_resnorm_bwd(None, y, y, None, torch.zeros(4, rows, device=DEV), gate=g,
                                        gate_act=act, pre_norm=False, sync=True)
        leaf = g.double().requires_grad_()
        a = ref.ACT[act](leaf)
        want = a.detach().expand(rows, H)
        tol = UNITS[act] * 2.0 ** -23 * want.abs() + 2.0 ** -148
        assert bool(((got.dy.double() - want).abs() <= tol).all())
        slope, = torch.autograd.grad(a.expand(rows, H).sum(), leaf)
        times = rows * H / g.numel()
        assert bool(((got.dgate.double() - slope).abs() <= 2.0 ** -19 * times).all())


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
def test_bf16_gates_far_from_zero(cuda_lib, act):
    """Every bf16 gate, forward and backward: the faster exponential that bf16 rows may take is off
    by at most 2 + 1.2 |g| units, with the rest 2^-16 of a normal result; half a step of bf16 is
    2^-8 of it, or 2^-134."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF).to(DEV).view(128, 512)
    y = torch.ones(128, 512, dtype=BF, device=DEV)
    want = ref.ACT[act](every.double())
    nan = want.isnan()
    kw = dict(gate=every, gate_act=act, pre_norm=False, sync=True)
    got, _, stats = cuda_lib.flce_resnorm_fwd(y, **kw)
    g = cuda_lib.flce_resnorm_bwd(None, y, y, None, stats, **kw)
    for v in (got, g.dy):
        assert torch.equal(v.isnan(), nan)
        err = (v.double() - want).abs()[~nan]
        assert bool((err <= (2.0 ** -8 + 2.0 ** -16) * want[~nan].abs() + 2.0 ** -134).all())


# ----------------------------------------------------------------------- modules
def _off(t, n=1):
    """t's values `n` elements behind a 16-byte boundary."""
    raw = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    v = raw[n:n + t.numel()].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gate", [(), (64,), (24, 1), (24, 64)])
def test_modules_take_views_at_any_element(cuda_lib, dtype, gate):
    """Inputs, parameters, incoming gradients that begin anywhere in a flat buffer: the bits of the
    same call on tensors of their own."""
    flce, N, H = cuda_lib, 24, 64
    t = dict(y=_randn(N, H, dtype=dtype, seed=1), h=_randn(N, H, dtype=dtype, seed=2),
             gate=_randn(*gate, dtype=dtype),
             **{k: _randn(H, dtype=dtype, seed=i) for i, k in
                enumerate(("w_pre", "b_pre", "w_post", "b_post"))})
    grads = [_randn(N, H, dtype=dtype, seed=3), _randn(N, H, dtype=dtype, seed=4)]
    join = flce.ResidualNorm("layer", gate_act="tanh")

    def run(place):
        leaves = {k: place(v).requires_grad_() for k, v in t.items()}
        kw = dict(leaves)
        out = join(kw.pop("y"), kw.pop("h"), **kw)
        g = torch.autograd.grad(out, list(leaves.values()), [place(x) for x in grads])
        return [*out, *g]

    for a, b in zip(run(_off), run(torch.clone)):
        assert torch.equal(a, b)


def test_linear_takes_views_at_any_element(cuda_lib):
    """Small whole numbers, which every product here holds exactly."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x, W, dy = (torch.randint(-2, 3, s, generator=g, device=DEV).to(BF)
                for s in ((24, 64), (48, 64), (24, 48)))

    def run(place):
        leaves = [place(v).requires_grad_() for v in (x, W)]
        out = cuda_lib.CheckpointedLinear()(*leaves)
        return [out, *torch.autograd.grad(out, leaves, place(dy))]

    for a, b in zip(run(_off), run(torch.clone)):
        assert torch.equal(a, b)


class _Saved:
    """The tensors that autograd keeps between the passes."""

    def __enter__(self):
        self.kept = []

        def pack(t):
            self.kept.append(t)
            return t

        self.hooks = torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t)
        self.hooks.__enter__()
        return self

    def __exit__(self, *a):
        self.hooks.__exit__(*a)

    def holds(self, t):
        return any(k.data_ptr() == t.data_ptr() for k in self.kept)


@pytest.mark.parametrize("kw,y_needed,h_needed", [
    (dict(), False, True), (dict(w_post=True), True, True), (dict(gate=True), True, True),
    (dict(pre_norm=False), False, False), (dict(pre_norm=False, w_post=True), True, False)])
def test_join_keeps_what_its_gradients_read(cuda_lib, kw, y_needed, h_needed):
    N, H = 40, 264
    kw = dict(kw)
    y, h = _randn(N, H, seed=1).requires_grad_(), _randn(N, H, seed=2).requires_grad_()
    p = {k: _randn(H, seed=3).requires_grad_() for k in ("w_post", "gate") if kw.pop(k, False)}
    opts = dict(kind="rms", gate_act=None, alpha=1.0, beta=1.0, eps=1e-6,
                pre_norm=kw.get("pre_norm", True), post_norm="w_post" in p)
    with _Saved() as saved:
        ho, z = cuda_lib.ResidualNorm(**kw)(y, h, **p)
    assert saved.holds(y) == y_needed and saved.holds(ho) == h_needed
    dz = _randn(N, H, seed=4) if opts["pre_norm"] else None
    dh_out = _randn(N, H, seed=5)
    leaves = dict(dy=y, dh=h, **{"d" + k: v for k, v in p.items()})
    outs = [(ho, dh_out)] + ([(z, dz)] if dz is not None else [])
    got = torch.autograd.grad([o for o, _ in outs], list(leaves.values()), [g for _, g in outs])
    want = ref.join_grads(dz, dh_out, y.detach(), ho.detach(),
                          {k: p[k].detach() if k in p else None
                           for k in ("w_pre", "b_pre", "w_post", "b_post", "gate")}, opts)
    for (k, leaf), g in zip(leaves.items(), got):
        ref.check(g, *want[k], k)


def test_gradients_without_y(cuda_lib):
    """The entry point itself takes no y where nothing reads it, and says so where something does."""
    N, H = 40, 264
    y, h, dz, dh = (_randn(N, H, seed=i) for i in range(4))
    out, _, stats = cuda_lib.flce_resnorm_fwd(y, h)
    full = cuda_lib.flce_resnorm_bwd(dz, dh, y, out, stats)
    for args in ((dz, dh), (dz, None)):
        a = cuda_lib.flce_resnorm_bwd(*args, None, out, stats, sync=True)
        b = cuda_lib.flce_resnorm_bwd(*args, y, out, stats)
        assert torch.equal(a.dy, b.dy) and torch.equal(a.dh, b.dh)
    assert torch.equal(full.dy, cuda_lib.flce_resnorm_bwd(dz, dh, None, out, stats).dy)
    only = cuda_lib.flce_resnorm_bwd(None, dh, None, None, stats, pre_norm=False, sync=True)
    assert torch.equal(only.dy, dh) and torch.equal(only.dh, dh)
    mixed = cuda_lib.flce_resnorm_bwd(None, dh.float(), None, None, stats, pre_norm=False,
                                      dtype=BF, sync=True)
    assert torch.equal(mixed.dy, dh) and torch.equal(mixed.dh, dh.float())
    for kw in (dict(post_norm=True), dict(gate=_randn(H))):
        with pytest.raises(ValueError):
            cuda_lib.flce_resnorm_bwd(dz, dh, None, out, stats, **kw)
    with pytest.raises(ValueError):
        cuda_lib.flce_resnorm_bwd(None, None, None, None, stats, pre_norm=False)


def test_linear_keeps_no_checkpoint_without_a_use(cuda_lib, monkeypatch):
    """A weight that is frozen, and a call under no_grad."""
    import linear_cross_entropy_fwd_gb300.block as block
    calls, save = [], block.flce_ckpt_save
    monkeypatch.setattr(block, "flce_ckpt_save", lambda *a, **k: calls.append(1) or save(*a, **k))
    x, W = _randn(24, 64).requires_grad_(), _randn(48, 64)
    linear = cuda_lib.CheckpointedLinear()
    with _Saved() as saved:
        out = linear(x, W)
    assert not calls and all(t.dtype is not torch.uint8 for t in saved.kept)
    dy = _randn(24, 48)
    dx, = torch.autograd.grad(out, x, dy)
    assert torch.equal(dx, dy @ W)
    with torch.no_grad():
        assert torch.equal(linear(x, W.clone().requires_grad_()), x @ W.t())
    assert not calls
    ck = cuda_lib.flce_ckpt_save(x.detach())
    with _Saved() as saved:
        linear(x, W, ck)
    assert not saved.holds(ck.data)
    linear(x, W.clone().requires_grad_())
    assert len(calls) == 1


def test_unused_z_brings_nothing(cuda_lib):
    """Rows of the stream that are not finite, and a loss that does not go through z: dh is
    alpha dh_out and dy act(gate) dh_out, in those rows too; the pre-norm's parameters get zeros."""
    N, H = 24, 64
    y, h = _randn(N, H, dtype=FP, seed=1), _randn(N, H, dtype=FP, seed=2)
    h[3, 5], h[7, 0] = float("inf"), float("nan")
    y.requires_grad_(), h.requires_grad_()
    gate = _randn(H, dtype=FP, seed=3)
    w, b = _randn(H, dtype=FP).requires_grad_(), _randn(H, dtype=FP).requires_grad_()
    ho, _ = cuda_lib.ResidualNorm(alpha=0.5)(y, h, w_pre=w, b_pre=b, gate=gate)
    dh = _randn(N, H, dtype=FP, seed=4)
    ho.backward(dh)
    assert torch.equal(h.grad, 0.5 * dh) and torch.equal(y.grad, gate * dh)
    assert not w.grad.any() and not b.grad.any()


def test_linear_refuses_in_the_forward_pass(cuda_lib):
    """A weight larger than the gradient's entry point takes, or without rows or columns, and a
    checkpoint or a weight elsewhere than x.  A frozen weight needs no such gradient."""
    linear = cuda_lib.CheckpointedLinear()
    x = _randn(2, 8)
    for shape, y in (((1 << 20) + 8, 8), x), ((0, 8), x), ((8, 0), x[:, :0]):
        W = torch.zeros(shape, dtype=BF, device=DEV)
        assert linear(y, W).shape == (2, shape[0])
        with pytest.raises(ValueError):
            linear(y, W.requires_grad_())
    W = _randn(8, 8).requires_grad_()
    with pytest.raises(ValueError):
        linear(x, W, SimpleNamespace(N=2, H=8, data=torch.zeros(72, dtype=torch.uint8)))
    for a, b in ((x, W.detach().cpu()), (x.cpu(), W), (x.cpu(), W.detach().cpu())):
        with pytest.raises(ValueError):
            linear(a, b)


# ------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("dt,st", [(BF, BF), (BF, FP), (FP, FP)])
@pytest.mark.parametrize("post,gate,kind", [(False, None, "rms"), (True, "channel", "rms"),
                                            (True, "full", "layer")])
def test_checkpoint_of_many_rows(cuda_lib, dt, st, post, gate, kind):
    """Where each group of warps has many rows, pairs of rows among them, and where rows are
    asked for late (the sizes with most rows): the bytes of the definition for z's first and last
    rows, and those that a checkpoint of the stored z has for all."""
    for N, H in ((20011, 64), (9001, 200), (97301, 264), (3001, 1000), (1001, 5000), (6101, 8192),
                 (333, 8200)):
        p = dict(w_pre=_randn(H, dtype=dt, seed=1), kind=kind)
        if post:
            p["w_post"] = _randn(H, dtype=dt, seed=2)
        if gate is not None:
            p["gate"] = _randn(*((H,) if gate == "channel" else (N, H)), dtype=dt, seed=3)
        y, h = _randn(N, H, dtype=dt, seed=4), _randn(N, H, dtype=st, seed=5)
        ck = cuda_lib.Checkpoint.empty(N, H, DEV)
        ck.data.fill_(0xA5)
        out, z, stats = cuda_lib.flce_resnorm_fwd(y, h, **p, checkpoint=ck, sync=True)
        plain = cuda_lib.flce_resnorm_fwd(y, h, **p)
        assert all(torch.equal(a, b) for a, b in zip(plain, (out, z, stats)))
        assert torch.equal(ck.data, cuda_lib.flce_ckpt_save(z).data)
        P = 32 * math.ceil(H / 32)
        rows = torch.cat([torch.arange(5), torch.arange(N - 5, N)])
        codes, scales = ref.quantise(z[rows.to(DEV)])
        assert torch.equal(ck.data[:N * P].view(N, P)[rows.to(DEV)].cpu(), codes)
        assert torch.equal(ck.data[N * P:].view(N, -1)[rows.to(DEV)].cpu(), scales)


@pytest.mark.parametrize("N,O,I", [(16384, 1024, 4864), (16384, 1024, 2432)])
def test_wgrad_adds_pieces(cuda_lib, N, O, I):
    """A sum of one sign over many tokens, in 76 tiles of 256 or 128 columns that a CTA pair each
    does from end to end.  An accumulator takes 2048 tokens, 16 at a time; what a step cuts off is
    less than 2^-23 of the sum so far, k / 128 of the piece's after k steps: 64.5 2^-23 of a piece.
    Eight pieces are added with a rounding of 2^-24 each.  In one accumulator 1024 steps would cut
    off up to 512.5 2^-23, and half a unit on average: four times what is allowed."""
    g = torch.Generator(device=DEV).manual_seed(I)
    dY = torch.rand(N, O, generator=g, device=DEV).to(BF)
    ck = cuda_lib.flce_ckpt_save(torch.rand(N, I, generator=g, device=DEV).to(BF))
    dW = cuda_lib.flce_ckpt_wgrad(dY, ck, sync=True)
    want = dY.double().t() @ cuda_lib.flce_ckpt_load(ck).double()
    err = (dW.double() - want).norm() / want.norm()
    assert err <= 64.5 * 2.0 ** -23 + 8 * 2.0 ** -24
