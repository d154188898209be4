"""What is measured of the operators between a model's blocks, and their plain forms.

Two groups, what a block of a model needs besides its attention and its products:

  resnorm_fwd, resnorm_bwd   the residual join: the norm after a block, its gate and residual
                             scales, the sum into the residual stream, and the norm before the
                             next block; and the gradients of all of it
  ckpt, wgrad                activation checkpoints in 8 bits: storing and reading back, and the
                             weight gradient of a projection taken from the stored input

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with
``own`` true it calls the package's entry points on the same data.  ``exact`` computes them in
64 bits from the definitions.

A checkpoint's buffer holds e4m3 codes [N, P] with P = 32 ceil(H / 32), then scale bytes
[N, 4 ceil(P / 128)]: 32 values of a row share the power of two 2^(byte - 127).
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases
def _join(op, N, H, dtype="bf16", stream="bf16", kind="rms", post=False, bias=False, gate="none",
          act="none", alpha=1.0, beta=1.0, params="bf16"):
    return {"op": op, "N": N, "H": H, "dtype": dtype, "stream": stream, "kind": kind,
            "post": post, "bias": bias, "gate": gate, "act": act, "alpha": alpha, "beta": beta,
            "params": params}


def listed():
    return [
        # one token of one user at the head's hidden size: all latency
        {"name": "resnorm_fwd_1_token", **_join("resnorm_fwd", 1, 4096)},
        # the 8192-token batch of the benchmark, norms on both sides of the block and a
        # learned gate per channel
        {"name": "resnorm_fwd_sandwich", **_join("resnorm_fwd", 8192, 4096, post=True,
                                                 gate="channel")},
        # an fp32 stream beside bf16 blocks, layer norms with biases, a computed gate per element
        {"name": "resnorm_fwd_layer_odd", **_join("resnorm_fwd", 3001, 1000, stream="fp32",
                                                  kind="layer", post=True, bias=True,
                                                  gate="full", act="sigmoid", params="fp32")},
        # its backward pass: the benchmark's batch
        {"name": "resnorm_bwd_sandwich", **_join("resnorm_bwd", 8192, 4096, post=True,
                                                 gate="channel")},
        # fp32 throughout, odd sizes, one gate per token, scaled residuals
        {"name": "resnorm_bwd_fp32_odd", **_join("resnorm_bwd", 1994, 2056, dtype="fp32",
                                                 stream="fp32", kind="layer", bias=True,
                                                 gate="token", act="tanh", alpha=1.5, beta=0.7,
                                                 params="fp32")},
        # the long-context batch: a plain pre-norm block
        {"name": "resnorm_bwd_long_context", **_join("resnorm_bwd", 65536, 4096)},
        # checkpoint of a small evaluation batch in fp32, odd width
        {"name": "ckpt_small_odd", "op": "ckpt", "N": 57, "H": 1000, "dtype": "fp32"},
        # checkpoint of the long-context batch
        {"name": "ckpt_long_context", "op": "ckpt", "N": 65536, "H": 4096, "dtype": "bf16"},
        # weight gradient over a ragged batch, narrow projection of odd sizes
        {"name": "wgrad_small_odd", "op": "wgrad", "N": 1994, "O": 1000, "I": 2056,
         "accumulate": False},
        # the small head's hidden size, added to what earlier micro-batches left
        {"name": "wgrad_2048_accumulate", "op": "wgrad", "N": 2048, "O": 2048, "I": 2048,
         "accumulate": True},
        # query, key and value projection of 32 / 8 heads of 128, the 8192-token batch
        {"name": "wgrad_qkv", "op": "wgrad", "N": 8192, "O": 6144, "I": 4096,
         "accumulate": False},
        # an up-projection over a batch of long documents
        {"name": "wgrad_up", "op": "wgrad", "N": 16384, "O": 14336, "I": 4096,
         "accumulate": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["resnorm_fwd", "resnorm_bwd", "resnorm_bwd", "ckpt", "wgrad"])
    if op == "ckpt":
        H = 8 * _log_int(rng, 8, 1024)
        return {"op": op, "N": min(_log_int(rng, 1, 65536), (1 << 27) // H), "H": H,
                "dtype": rng.choice(["bf16", "fp32"])}
    if op == "wgrad":
        O, I = 8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 8, 1024)
        return {"op": op, "N": min(_log_int(rng, 1, 16384), int(1.6e11 / (O * I))), "O": O,
                "I": I, "accumulate": rng.choice([False, True])}
    H = 8 * _log_int(rng, 8, 1024)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    gate = rng.choice(["none", "channel", "token", "full", "scalar"])
    return _join(op, min(_log_int(rng, 1, 65536), (1 << 26) // H), H, dtype=dtype,
                 stream="fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"]),
                 kind=rng.choice(["rms", "layer"]), post=rng.choice([False, True]),
                 bias=rng.choice([False, True]), gate=gate,
                 act="none" if gate == "none" else rng.choice(["none", "sigmoid", "tanh"]),
                 alpha=rng.choice([1.0, 1.5]), beta=rng.choice([1.0, 0.25]),
                 params="fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"]))


# ----------------------------------------------------------------- inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _activations(g, N, H, dtype):
    """Activations: tokens of different sizes, and about one channel in a hundred that
    stands far out."""
    x = _randn(g, N, H) * torch.exp(_randn(g, N, 1, std=0.5))
    loud = torch.rand(H, generator=g, device="cuda") < 0.01
    return torch.where(loud[None, :], 20.0 * x, x).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "ckpt":
        s["x"] = _activations(g, case["N"], case["H"], _dt(case["dtype"]))
        return s
    if op == "wgrad":
        s["dY"] = _randn(g, case["N"], case["O"], dtype=torch.bfloat16)
        s["ckpt"] = _encode(_activations(g, case["N"], case["I"], torch.bfloat16))
        # what earlier micro-batches left in the weight's gradient
        s["dW"] = _randn(g, case["O"], case["I"], std=30.0) if case["accumulate"] else None
        return s
    N, H, dt, st, pt = (case["N"], case["H"], _dt(case["dtype"]), _dt(case["stream"]),
                        _dt(case["params"]))
    s["y"] = _activations(g, N, H, dt)
    s["h"] = _randn(g, N, H, dtype=st, std=3.0)
    for n in ("pre", "post") if case["post"] else ("pre",):
        s["w_" + n] = (1.0 + _randn(g, H, std=0.2)).to(pt)
        if case["bias"]:
            s["b_" + n] = _randn(g, H, dtype=pt, std=0.1)
    shape = {"channel": (H,), "token": (N, 1), "full": (N, H), "scalar": ()}
    if case["gate"] != "none":
        # a learned gate is a parameter, one computed for each token an activation
        s["gate"] = ((0.5 + _randn(g, *shape[case["gate"]], std=0.5))
                     .to(pt if case["gate"] in ("channel", "scalar") else dt))
    if op == "resnorm_bwd":
        h, z, stats = _plain_fwd(s)
        s.update(h_out=h, stats=stats)
        del s["h"], h
        s["dz"] = _randn(g, *z.shape, dtype=dt)
        # the stream's gradient leans on what the block added to it
        s["dh_out"] = (_randn(g, N, H) + 0.3 * s["y"].float()).to(st)
    return s


# ------------------------------------------------------------ plain forms
def _normalised(x, layer):
    """(x - mean) / sqrt(var + eps), with mean and 1 / sqrt; the mean is 0 unless `layer`."""
    mean = x.mean(1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    x = x - mean
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    return x * r, mean, r


def _affine(x, w, b):
    if w is not None:
        x = x * w.float()
    return x if b is None else x + b.float()


def _gate(s):
    """act(gate) and its derivative, in 32 bits."""
    if "gate" not in s:
        return None, None
    g, act = s["gate"].float(), s["case"]["act"]
    if act == "none":
        return g, torch.ones_like(g)
    if act == "sigmoid":
        a = 1.0 / (1.0 + torch.exp(-g))
        return a, a * (1.0 - a)
    a = torch.tanh(g)
    return a, 1.0 - a * a


def _plain_fwd(s):
    c = s["case"]
    layer = c["kind"] == "layer"
    zeros = torch.zeros(c["N"], 1, device="cuda")
    u, mean_y, r_y = s["y"].float(), zeros, zeros
    if c["post"]:
        u, mean_y, r_y = _normalised(u, layer)
        u = _affine(u, s.get("w_post"), s.get("b_post"))
    a, _ = _gate(s)
    h = c["alpha"] * s["h"].float() + c["beta"] * (u if a is None else a * u)
    # the stream is what is stored of it: the norm and the gradients take it as it is read back
    h = h.to(s["h"].dtype)
    z, mean_h, r_h = _normalised(h.float(), layer)
    z = _affine(z, s.get("w_pre"), s.get("b_pre"))
    stats = torch.cat([mean_y, r_y, mean_h, r_h], 1).t().contiguous()
    return h, z.to(s["y"].dtype), stats


def _norm_gradient(g, xh, r, layer):
    g2 = g - xh * (g * xh).mean(1, keepdim=True)
    return r * (g2 - g.mean(1, keepdim=True) if layer else g2)


def _plain_bwd(s):
    c, out = s["case"], {}
    layer = c["kind"] == "layer"
    mean_y, r_y, mean_h, r_h = (x[:, None] for x in s["stats"])
    xh = (s["h_out"].float() - mean_h) * r_h
    dz = s["dz"].float()
    out["dw_pre"] = (dz * xh).sum(0)
    if c["bias"]:
        out["db_pre"] = dz.sum(0)
    dt = _norm_gradient(dz * s["w_pre"].float(), xh, r_h, layer) + s["dh_out"].float()
    del xh, dz
    out["dh"] = (c["alpha"] * dt).to(s["dh_out"].dtype)
    a, slope = _gate(s)
    du = c["beta"] * (dt if a is None else a * dt)
    y = s["y"].float()
    yh = (y - mean_y) * r_y if c["post"] else y
    if a is not None:
        u = _affine(yh, s.get("w_post"), s.get("b_post")) if c["post"] else yh
        dg = c["beta"] * slope * u * dt
        # gradients of parameters are fp32, those of activations have their type
        out["dgate"] = {"channel": lambda: dg.sum(0), "scalar": lambda: dg.sum(),
                        "token": lambda: dg.sum(1, keepdim=True).to(s["gate"].dtype),
                        "full": lambda: dg.to(s["gate"].dtype)}[c["gate"]]()
    if c["post"]:
        out["dw_post"] = (du * yh).sum(0)
        if c["bias"]:
            out["db_post"] = du.sum(0)
        du = _norm_gradient(du * s["w_post"].float(), yh, r_y, layer)
    out["dy"] = du.to(s["y"].dtype)
    return out


def _groups(x):
    """x in 32 bits as [N, groups, 32], zeros behind a row's end, and each group's scale."""
    N, H = x.shape
    P = 32 * -(-H // 32)
    full = torch.zeros(N, P, device=x.device)
    full[:, :H] = x
    full = full.view(N, P // 32, 32)
    m, e = torch.frexp(full.abs().amax(2, keepdim=True))  # m in [0.5, 1), 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, -117), e).clamp(-117, 119)
    return full, e


def _pow2(e):
    """2^e for whole e of the normal range."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _plain_ckpt(x):
    full, e = _groups(x)
    v = full * _pow2(-e)
    # a value of e4m3 has steps of 2^-3 of its power of two, and 2^-9 at the least
    _, k = torch.frexp(v)
    step = _pow2((k - 4).clamp(min=-9))
    v = torch.round(v / step) * step
    return (v * _pow2(e)).view(x.shape[0], -1)[:, :x.shape[1]].to(x.dtype)


def _encode(x):
    """A checkpoint of x as its bytes."""
    N = x.shape[0]
    full, e = _groups(x)
    codes = (full * _pow2(-e)).to(torch.float8_e4m3fn).view(torch.uint8).view(N, -1)
    scales = torch.zeros(N, 4 * -(-codes.shape[1] // 128), dtype=torch.uint8, device="cuda")
    scales[:, :e.shape[1]] = (e[:, :, 0] + 127).to(torch.uint8)
    return torch.cat([codes.reshape(-1), scales.reshape(-1)])


def _plain_decode(buf, N, H):
    """The values that a checkpoint's bytes stand for, in 32 bits."""
    P = 32 * -(-H // 32)
    code = buf[:N * P].view(N, P // 32, 32).int()
    scale = buf[N * P:].view(N, -1)[:, :P // 32, None].int()
    e, m = code >> 3 & 15, (code & 7).float()
    v = torch.where(e > 0, (8 + m) * _pow2(e - 10), m * 2.0 ** -9)
    v = torch.where(code > 127, -v, v) * _pow2(scale - 127)
    return v.view(N, P)[:, :H]


def _plain_wgrad(s):
    c = s["case"]
    x = _plain_decode(s["ckpt"], c["N"], c["I"])
    dW = s["dY"].float().t() @ x
    return dW if s["dW"] is None else s["dW"].add_(dW)


# -------------------------------------------------------------------- run
def run(state):
    op, c = state["op"], state["case"]
    if not own:
        if op == "resnorm_fwd":
            h, z, _ = _plain_fwd(state)
            return {"h": h, "z": z}
        if op == "resnorm_bwd":
            return _plain_bwd(state)
        return _plain_ckpt(state["x"]) if op == "ckpt" else _plain_wgrad(state)
    import linear_cross_entropy_fwd_gb300 as flce
    s = state
    if op == "ckpt":
        return flce.flce_ckpt_load(flce.flce_ckpt_save(s["x"]), dtype=s["x"].dtype)
    if op == "wgrad":
        ckpt = flce.Checkpoint(s["ckpt"], c["N"], c["I"])
        return flce.flce_ckpt_wgrad(s["dY"], ckpt, dW=s["dW"], accumulate=c["accumulate"])
    kw = dict(w_pre=s["w_pre"], b_pre=s.get("b_pre"), w_post=s.get("w_post"),
              b_post=s.get("b_post"), gate=s.get("gate"), gate_act=c["act"], kind=c["kind"],
              alpha=c["alpha"], beta=c["beta"], eps=EPS)
    if op == "resnorm_fwd":
        h, z, _ = flce.flce_resnorm_fwd(s["y"], s["h"], **kw)
        return {"h": h, "z": z}
    g = flce.flce_resnorm_bwd(s["dz"], s["dh_out"], s["y"], s["h_out"], s["stats"], **kw)
    return {k: v for k, v in g._asdict().items() if v is not None}


# ------------------------------------------------------------------- work
def work(case):
    op, N = case["op"], case["N"]
    if op == "ckpt":
        H = case["H"]
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * N * H * (e + 1 + 1 / 32), "flops": 6 * N * H}
    if op == "wgrad":
        O, I = case["O"], case["I"]
        return {"bytes": N * (2 * O + I + I / 32) + O * I * (8 if case["accumulate"] else 4),
                "flops": 2.0 * N * O * I}
    H = case["H"]
    e, t, p = (2 if case[k] == "bf16" else 4 for k in ("dtype", "stream", "params"))
    rows = (1 + case["post"]) * (1 + case["bias"]) + (case["gate"] == "channel")
    full = {"full": N * H, "token": N}.get(case["gate"], 0)
    if op == "resnorm_fwd":
        return {"bytes": N * H * 2 * (e + t) + e * full + p * rows * H, "flops": 14 * N * H}
    return {"bytes": N * H * 3 * (e + t) + 2 * e * full + (p + 4) * rows * H + 16 * N,
            "flops": 30 * N * H}


# ---------------------------------------------------- 64 bits, definitions
def _exact_norm(x, s, name):
    c = s["case"]
    if c["kind"] == "layer":
        x = x - x.mean(1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    if "w_" + name in s:
        x = x * s["w_" + name]
    return x + s["b_" + name] if "b_" + name in s else x


def _exact_add(s):
    """beta act(gate) u of the join."""
    c, u = s["case"], s["y"]
    if c["post"]:
        u = _exact_norm(u, s, "post")
    if "gate" in s:
        u = u * {"none": lambda x: x, "sigmoid": torch.sigmoid,
                 "tanh": torch.tanh}[c["act"]](s["gate"])
    return c["beta"] * u


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ckpt":
        N, H = s["x"].shape
        x = torch.zeros(N, 32 * -(-H // 32), dtype=torch.float64, device="cuda")
        x[:, :H] = s["x"]
        x = x.view(N, -1, 32)
        top = x.abs().amax(2, keepdim=True).clamp(min=2.0 ** -140)
        e = torch.ceil(torch.log2(top / 448)).clamp(-117, 119)  # of a value within a border's
        e = torch.where(448 * torch.exp2(e) < top, e + 1, e)    # rounding, made sure of
        e = torch.where(448 * torch.exp2(e - 1) >= top, e - 1, e).clamp(-117, 119)
        v = x / torch.exp2(e)
        k = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -9))).clamp(min=-6)
        k = torch.where(torch.exp2(k) > v.abs(), (k - 1).clamp(min=-6), k)
        step = torch.exp2(k - 3)
        v = torch.round(v / step) * step * torch.exp2(e)
        return v.view(N, -1)[:, :H].contiguous()
    if op == "wgrad":
        N, I = case["N"], case["I"]
        P = 32 * -(-I // 32)
        codes = s["ckpt"][:N * P].view(torch.float8_e4m3fn).view(N, P).double()
        scales = s["ckpt"][N * P:].view(N, -1).double() - 127
        x = (codes * torch.exp2(scales).repeat_interleave(32, 1)[:, :P])[:, :I]
        out = s["dY"].double().t() @ x
        return out if s["dW"] is None else out + s["dW"].double()
    for k, v in s.items():
        if torch.is_tensor(v):
            s[k] = v.double()
    if op == "resnorm_fwd":
        h = case["alpha"] * s["h"] + _exact_add(s)
        return {"h": h, "z": _exact_norm(h.to(_dt(case["stream"])).double(), s, "pre")}
    names = [k for k in ("y", "w_post", "b_post", "gate", "h_out", "w_pre", "b_pre") if k in s]
    for k in names:
        s[k].requires_grad_()
    z = _exact_norm(s["h_out"], s, "pre")
    pre = [k for k in ("h_out", "w_pre", "b_pre") if k in s]
    got = dict(zip(pre, torch.autograd.grad(z, [s[k] for k in pre], s["dz"])))
    dt = got.pop("h_out") + s["dh_out"]
    del z
    rest = [k for k in names if k not in pre]
    got.update(zip(rest, torch.autograd.grad(_exact_add(s), [s[k] for k in rest], dt)))
    got["h"] = case["alpha"] * dt
    return {"d" + k: v for k, v in got.items()}
