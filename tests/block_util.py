"""The residual join and the 8-bit checkpoint in plain 64-bit torch, for the tests.

``join`` and ``join_grads`` return values and, beside each, a bound on what rounding in fp32 may
take it off by: U = 2^-24 times the sum of the magnitudes that went into it, times ROUNDS.  A
value passes at most 5 additions in a lane's butterfly, 8 in a thread, 16 across warps and 4
across a cluster on its way through a sum, the statistic is used in a product or two, each
operation rounds once, and the functions (rsqrt, exp, tanh, division) are within 2 units:
below 64 in all.  Sums over tokens round once more per token and part."""
import torch

U = 2.0 ** -24
ROUNDS = 64.0
ACT = {None: lambda g: g, "none": lambda g: g, "sigmoid": torch.sigmoid, "tanh": torch.tanh}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, want, bound, what):
    """|got - want| within half a step of got's type and the bound."""
    err = (got.double() - want).abs()
    tol = half_step(got.dtype) * want.abs() + bound
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err[bad].max()),
                                 float((err / tol).nan_to_num(1e9).max()))


def norm(x, kind, eps, w, b):
    """n(x) * w + b, the magnitude that its rounding goes by, and n(x)'s parts."""
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    r = (((x - mean) ** 2).mean(1, keepdim=True) + eps) ** -0.5
    xh = (x - mean) * r
    mag = (x.abs() + (x.abs().mean(1, keepdim=True) if kind == "layer" else 0)) * r
    out, size = xh, mag
    if w is not None:
        out, size = out * w, size * w.abs()
    if b is not None:
        out, size = out + b, size + b.abs()
    return out, size, xh, mag, r


def _d(t):
    return None if t is None else t.double()


def join(y, h, p, opts):
    """h_out before its rounding, with the bound of its fp32 arithmetic."""
    y, h = _d(y), _d(h)
    u, size = y, y.abs()
    if opts["post_norm"]:
        u, size, *_ = norm(y, opts["kind"], opts["eps"], _d(p["w_post"]), _d(p["b_post"]))
    if p["gate"] is not None:
        a = ACT[opts["gate_act"]](_d(p["gate"]))
        u, size = a * u, size * a.abs()
    out, size = opts["beta"] * u, abs(opts["beta"]) * size
    if h is not None:
        out, size = out + opts["alpha"] * h, size + abs(opts["alpha"]) * h.abs()
    return out, ROUNDS * U * size


def pre(h_out, p, opts):
    """z of the stored stream."""
    z, size, *_ = norm(_d(h_out), opts["kind"], opts["eps"], _d(p["w_pre"]), _d(p["b_pre"]))
    return z, ROUNDS * U * size


def join_grads(dz, dh_out, y, h_out, p, opts):
    """{name: (value, bound)} of the gradients at these inputs, from the formulas."""
    dz, dh_out, y, h_out = _d(dz), _d(dh_out), _d(y), _d(h_out)
    p = {k: _d(v) for k, v in p.items()}
    layer, eps = opts["kind"] == "layer", opts["eps"]
    N, H = y.shape
    one = torch.ones(H, dtype=torch.float64, device=y.device)
    per_token = (ROUNDS + N) * U
    out = {}
    dt, D = torch.zeros_like(y), torch.zeros_like(y)
    if dh_out is not None:
        dt, D = dh_out, dh_out.abs()
    if opts["pre_norm"]:
        _, _, xh, X, r = norm(h_out, opts["kind"], eps, None, None)
        w = p["w_pre"] if p["w_pre"] is not None else one
        g = dz * w
        dt = dt + r * (g - (g.mean(1, keepdim=True) if layer else 0)
                       - xh * (g * xh).mean(1, keepdim=True))
        G = g.abs()
        D = D + r * (G + (G.mean(1, keepdim=True) if layer else 0)
                     + X * (G * X).mean(1, keepdim=True))
        out["dw_pre"] = (dz * xh).sum(0), per_token * (dz.abs() * X).sum(0)
        out["db_pre"] = dz.sum(0), per_token * dz.abs().sum(0)
    out["dh"] = opts["alpha"] * dt, ROUNDS * U * abs(opts["alpha"]) * D
    yh, Y, r = y, y.abs(), 1.0
    if opts["post_norm"]:
        _, _, yh, Y, r = norm(y, opts["kind"], eps, None, None)
    w = p["w_post"] if p["w_post"] is not None else one
    u, size = yh * w, Y * w.abs()
    if p["b_post"] is not None:
        u, size = u + p["b_post"], size + p["b_post"].abs()
    a = torch.ones((), dtype=torch.float64, device=y.device)
    if p["gate"] is not None:
        gate = p["gate"].clone().requires_grad_()
        a = ACT[opts["gate_act"]](gate)
        slope, = torch.autograd.grad(a.sum(), gate)
        a = a.detach()
        dg, mag = opts["beta"] * slope * u * dt, abs(opts["beta"]) * size * D
        # a slope of fp32 is off by a unit of 1 where it is a difference of 1 and a product
        mag = mag * (slope.abs() + (0 if opts["gate_act"] in (None, "none") else 1))
        if gate.dim() == 0:
            out["dgate"] = dg.sum(), (ROUNDS + N * 16) * U * mag.sum()
        elif gate.dim() == 1:
            out["dgate"] = dg.sum(0), per_token * mag.sum(0)
        elif gate.shape[1] == 1:
            out["dgate"] = dg.sum(1, keepdim=True), ROUNDS * U * mag.sum(1, keepdim=True)
        else:
            out["dgate"] = dg, ROUNDS * U * mag
    du, S = opts["beta"] * a * dt, abs(opts["beta"]) * a.abs() * D
    if opts["post_norm"]:
        out["dw_post"] = (du * yh).sum(0), per_token * (S * Y).sum(0)
        out["db_post"] = du.sum(0), per_token * S.sum(0)
        gy, G = du * w, S * w.abs()
        du = r * (gy - (gy.mean(1, keepdim=True) if layer else 0)
                  - yh * (gy * yh).mean(1, keepdim=True))
        S = r * (G + (G.mean(1, keepdim=True) if layer else 0)
                 + Y * (G * Y).mean(1, keepdim=True))
    out["dy"] = du, ROUNDS * U * S
    return out


def quantise(x):
    """What a checkpoint of x [N, H] holds: codes [N, P] and scale bytes [N, S], from the
    definition, value by value against the table of e4m3 numbers."""
    N, H = x.shape
    P, S = 32 * -(-H // 32), 4 * -(-H // 128)
    full = torch.zeros(N, P, dtype=torch.float64)
    full[:, :H] = x.double().cpu()
    full = full.view(N, P // 32, 32)
    bad = ~torch.isfinite(full).all(2)
    full = torch.where(bad[..., None], torch.zeros_like(full), full)
    top = full.abs().amax(2)
    e = torch.full(top.shape, -117, dtype=torch.int64)
    for k in range(-116, 120):
        e = torch.where(top > 448 * 2.0 ** (k - 1), torch.full_like(e, k), e)
    v = torch.ldexp(full, -e[..., None])  # exact
    table = e4m3_table()[:127]            # the numbers 0 .. 448, ascending
    mid = (table[1:] + table[:-1]) / 2    # a tie goes to the even code
    code = torch.bucketize(v.abs(), mid, right=False)
    tie = (code < 126) & (v.abs() == mid[code.clamp(max=125)])
    code = torch.where(tie & (code % 2 == 1), code + 1, code)
    code = torch.where(torch.signbit(full), code + 128, code).to(torch.uint8)
    scales = torch.zeros(N, S, dtype=torch.uint8)
    scales[:, :P // 32] = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return code.view(N, P), scales


def e4m3_table():
    """The values of the codes 0 .. 255 (NaN at 127 and 255)."""
    c = torch.arange(256)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (8 + m) * 2.0 ** (e.double() - 10), m * 2.0 ** -9)
    v[(c & 127) == 127] = float("nan")
    return torch.where(c > 127, -v, v)


def dequantise(codes, scales, H):
    """The values that they stand for."""
    N, P = codes.shape
    s = scales[:, :P // 32].double()
    f = torch.where(s == 255, torch.full_like(s, float("nan")), 2.0 ** (s - 127))
    return (e4m3_table()[codes.long()].view(N, P // 32, 32) * f[..., None]).view(N, P)[:, :H]
