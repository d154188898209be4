"""What is measured of the operators around the linear cross-entropy head, and their plain forms.

Three groups, the parts of one training step that stand next to the head:

  embed_fwd, embed_bwd   embedding lookup with a scale, and its gradient (dense, or added to
                         the gradient that the head left in a tied weight)
  attn_fwd, attn_train   causal attention over packed sequences with grouped heads: the
                         forward pass, and the forward pass followed by the gradients
  orthogonalize          Newton-Schulz iterations on an update matrix

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with
``own`` true it calls the package's entry points on the same data.  ``exact`` computes them in
64 bits from the definitions.
"""
import math

import torch

own = False

IGN = -100
COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a few users: the lookup is all latency
        {"name": "embed_fwd_8_tokens", "op": "embed_fwd", "N": 8, "H": 4096, "V": 128256,
         "dtype": "bf16", "scale": 1.0},
        # the long-context batch of the benchmark, embeddings scaled by sqrt(H)
        {"name": "embed_fwd_long_context", "op": "embed_fwd", "N": 65536, "H": 4096, "V": 128256,
         "dtype": "bf16", "scale": 64.0},
        # tied weight: the embedding's gradient joins the head's fp32 dW (8192-token batch)
        {"name": "embed_bwd_tied", "op": "embed_bwd", "N": 8192, "H": 4096, "V": 128256,
         "dtype": "bf16", "scale": 1.0, "accumulate": True},
        # untied weight in fp32, odd token count and vocabulary: the dense gradient
        {"name": "embed_bwd_dense_odd", "op": "embed_bwd", "N": 3001, "H": 1000, "V": 32003,
         "dtype": "fp32", "scale": 0.5, "accumulate": False},
        # a handful of short prompts, evaluation: latency
        {"name": "attn_fwd_short", "op": "attn_fwd", "lens": "57,1,130", "pad": 4, "Hq": 8,
         "Hkv": 2, "D": 64},
        # packed prompts of an 8192-token batch with the benchmark head's hidden size 4096
        {"name": "attn_fwd_prompts", "op": "attn_fwd", "lens": "4096,2311,1001,784", "pad": 0,
         "Hq": 32, "Hkv": 8, "D": 128},
        # a small training batch, many ragged sequences, an empty one among them
        {"name": "attn_train_ragged", "op": "attn_train",
         "lens": "333,128,0,700,65,1,255,512", "pad": 54, "Hq": 16, "Hkv": 4, "D": 64},
        # one training batch of long documents
        {"name": "attn_train_long", "op": "attn_train", "lens": "8192,5000,3100", "pad": 92,
         "Hq": 32, "Hkv": 8, "D": 128},
        # small projections of several layers, stacked
        {"name": "orthogonalize_stack", "op": "orthogonalize", "B": 8, "m": 256, "n": 1024,
         "dtype": "bf16"},
        # a square projection at the small head's hidden size
        {"name": "orthogonalize_2048", "op": "orthogonalize", "B": 1, "m": 2048, "n": 2048,
         "dtype": "fp32"},
        # a tall matrix of odd shape (rows > columns)
        {"name": "orthogonalize_tall_odd", "op": "orthogonalize", "B": 1, "m": 3584, "n": 1000,
         "dtype": "fp32"},
        # an up-projection at the Llama-3 head's hidden size
        {"name": "orthogonalize_wide", "op": "orthogonalize", "B": 1, "m": 4096, "n": 14336,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + (n in (384, 3072))  # neither a size of 3072 nor 8 * 384


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "attn_fwd", "attn_train", "orthogonalize"])
    if op in ("embed_fwd", "embed_bwd"):
        case = {"op": op, "N": _log_int(rng, 8, 65536), "H": 8 * _log_int(rng, 32, 512),
                "V": _log_int(rng, 4000, 128256), "dtype": rng.choice(["bf16", "fp32"]),
                "scale": rng.choice([0.5, 1.0, 45.25, 64.0])}
        if op == "embed_bwd":
            case["N"] = _log_int(rng, 8, 8192)
            case["accumulate"] = rng.choice([False, True])
        elif case["dtype"] == "fp32":
            case["N"] = min(case["N"], 32768)
        return case
    if op in ("attn_fwd", "attn_train"):
        top = 4096 if op == "attn_fwd" else 8192
        budget = 2.1e9 if op == "attn_fwd" else 4.0e9
        heads = rng.choice([(8, 2), (16, 4), (32, 8), (8, 8), (16, 1), (12, 4)])
        lens = [_log_int(rng, 1, top) for _ in range(rng.randint(1, 8))]
        if rng.random() < 0.3:
            lens[rng.randrange(len(lens))] = 0
        # a batch as dense [sequences, longest, longest] per head stays within the largest case
        while len(lens) * max(lens) ** 2 * heads[0] > budget or max(lens) == 0:
            lens = [max(1, n // 2) for n in lens]
        return {"op": op, "lens": ",".join(str(n) for n in lens), "pad": rng.choice([0, 0, 1, 37]),
                "Hq": heads[0], "Hkv": heads[1], "D": rng.choice([64, 64, 80, 128, 128])}
    m, n, b = _log_int(rng, 64, 4096), _log_int(rng, 64, 8192), rng.choice([1, 1, 2, 5])
    if rng.random() < 0.5:
        m, n = n, m
    if rng.random() < 0.5:
        m, n = (8 * -(-x // 8) + 8 * (3064 < x <= 3072) for x in (m, n))
    if m * n > 1 << 22:
        b = 1
    return {"op": op, "B": b, "m": m, "n": n, "dtype": rng.choice(["bf16", "fp32"])}


# ----------------------------------------------------------------- inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _ids(g, N, V):
    """Token ids whose frequencies fall like 1/rank, ranks spread over the table, and
    about one in fifty tokens ignored."""
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    ids = rank * 7919 % V
    drop = torch.rand(N, generator=g, device="cuda") < 0.02
    return torch.where(drop, torch.full_like(ids, IGN), ids)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "embed_fwd":
        s["W"] = _randn(g, case["V"], case["H"], dtype=_dt(case["dtype"]), std=0.02)
        s["ids"] = _ids(g, case["N"], case["V"])
    elif op == "embed_bwd":
        s["dY"] = _randn(g, case["N"], case["H"], dtype=_dt(case["dtype"]))
        s["ids"] = _ids(g, case["N"], case["V"])
        # a tied weight: what the head's backward pass left there
        s["dW"] = _randn(g, case["V"], case["H"]) if case["accumulate"] else None
    elif op in ("attn_fwd", "attn_train"):
        lens, Hq, Hkv, D = _lens(case), case["Hq"], case["Hkv"], case["D"]
        T = sum(lens) + case["pad"]
        # q, k and v are slices of one projection's output, as a model has them
        qkv = _randn(g, T, Hq + 2 * Hkv, D, dtype=torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        s["cu"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        s["longest"] = max(lens)
        if op == "attn_train":
            s["dO"] = _randn(g, T, Hq, D, dtype=torch.bfloat16)
    else:
        B, m, n = case["B"], case["m"], case["n"]
        # a momentum matrix: a few strong directions over a noise floor
        r = 16
        u = _randn(g, B, m, r) * torch.logspace(0, -1, r, device="cuda")
        s["G"] = ((u @ _randn(g, B, r, n)).mul_(0.3).add_(_randn(g, B, m, n))
                  .mul_(1e-3).to(_dt(case["dtype"])))
    return s


# ------------------------------------------------------------ plain forms
def _plain_embed_fwd(s):
    W, ids, c = s["W"], s["ids"], s["case"]
    rows = W[ids.clamp(min=0)].float() * c["scale"]
    return rows.masked_fill_((ids == IGN)[:, None], 0.0).to(W.dtype)


def _plain_embed_bwd(s):
    dY, ids, c = s["dY"], s["ids"], s["case"]
    dW = s["dW"]
    if dW is None:
        dW = torch.zeros(c["V"], c["H"], device="cuda")
    rows = (dY.float() * c["scale"]).masked_fill_((ids == IGN)[:, None], 0.0)
    return dW.index_add_(0, ids.clamp(min=0), rows)


def _plain_attn(s, train):
    """Each sequence is one row of a dense batch [sequences, longest]; places past a
    sequence's end are masked."""
    q, k, v, cu, L = s["q"], s["k"], s["v"], s["cu"].long(), s["longest"]
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    R, B = Hq // Hkv, cu.numel() - 1
    sc = 1.0 / math.sqrt(D)
    pos = torch.arange(L, device="cuda")
    inside = pos[None, :] < (cu[1:] - cu[:-1])[:, None]                    # [B, L]
    at = torch.where(inside, cu[:-1, None] + pos[None, :], torch.full_like(pos, T)[None, :])

    def dense(x):                                                          # [B, Hkv, R, L, D]
        x = torch.cat([x.float(), x.new_zeros(1, *x.shape[1:]).float()])[at]
        return x.view(B, L, Hkv, -1, D).permute(0, 2, 3, 1, 4)

    def packed(x, like):                                                   # back to [T, heads, D]
        out = torch.zeros(T + 1, *like.shape[1:], device="cuda")
        out[at.reshape(-1)] = x.permute(0, 3, 1, 2, 4).reshape(B * L, -1, like.shape[2])
        return out[:T].to(like.dtype)

    Q, K, V = dense(q).reshape(B, Hkv, R * L, D), dense(k)[:, :, 0], dense(v)[:, :, 0]
    S = torch.matmul(Q, K.transpose(2, 3)).mul_(sc).view(B, Hkv, R, L, L)
    S.masked_fill_(pos[None, :] > pos[:, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    P = S.sub_(m).exp_()
    l = P.sum(-1, keepdim=True)
    P.div_(l)
    O = torch.matmul(P.view(B, Hkv, R * L, L), V).view(B, Hkv, R, L, D)
    lse = torch.full((Hq, T + 1), -math.inf, device="cuda")
    lse[:, at.reshape(-1)] = (m + l.log())[..., 0].permute(1, 2, 0, 3).reshape(Hq, B * L)
    lse[:, T] = -math.inf
    out = {"o": packed(O, q), "lse": lse[:, :T].contiguous()}
    if not train:
        return out
    dO = dense(s["dO"])
    dOf = dO.reshape(B, Hkv, R * L, D)
    Pf = P.view(B, Hkv, R * L, L)
    dV = torch.matmul(Pf.transpose(2, 3), dOf)
    dP = torch.matmul(dOf, V.transpose(2, 3)).view(B, Hkv, R, L, L)
    dS = dP.sub_((dO * O).sum(-1, keepdim=True)).mul_(P).mul_(sc).view(B, Hkv, R * L, L)
    dQ = torch.matmul(dS, K).view(B, Hkv, R, L, D)
    dK = torch.matmul(dS.transpose(2, 3), Q)
    out.update(dq=packed(dQ, q), dk=packed(dK[:, :, None], k), dv=packed(dV[:, :, None], v))
    return out


def _plain_orthogonalize(s):
    a, b, c = COEFFS
    X = s["G"].float()
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    tall = X.shape[1] > X.shape[2]
    if tall:
        X = X.transpose(1, 2)

    def step(X):
        M = X @ X.transpose(1, 2)
        return a * X + (b * M + c * (M @ M)) @ X

    X = step(step(step(step(step(X)))))
    return (X.transpose(1, 2) if tall else X).to(torch.bfloat16).contiguous()


def run(state):
    op, c = state["op"], state["case"]
    if not own:
        if op == "embed_fwd":
            return _plain_embed_fwd(state)
        if op == "embed_bwd":
            return _plain_embed_bwd(state)
        if op == "orthogonalize":
            return _plain_orthogonalize(state)
        return _plain_attn(state, op == "attn_train")
    import linear_cross_entropy_fwd_gb300 as flce
    if op == "embed_fwd":
        return flce.flce_embed_fwd(state["W"], state["ids"], scale=c["scale"], ignore_index=IGN)
    if op == "embed_bwd":
        return flce.flce_embed_bwd(state["dY"], state["ids"], c["V"], scale=c["scale"],
                                   ignore_index=IGN, dW=state["dW"], accumulate=c["accumulate"])
    if op == "orthogonalize":
        return flce.flce_orthogonalize(state["G"], steps=5, coeffs=COEFFS, eps=EPS)
    q, k, v, cu = state["q"], state["k"], state["v"], state["cu"]
    o, lse = flce.flce_attn_fwd(q, k, v, cu)
    out = {"o": o, "lse": lse}
    if op == "attn_train":
        dq, dk, dv = flce.flce_attn_bwd(state["dO"], q, k, v, o, lse, cu)
        out.update(dq=dq, dk=dk, dv=dv)
    return out


# ------------------------------------------------------------------- work
def _unique(N, V):
    """Expected number of different ids among N drawn as _ids() draws them."""
    step = max(1, V // 4096)
    total = 0.0
    for r in range(1, V + 1, step):
        p = math.log((r + 1.0) / r) / math.log(V)
        total += min(step, V + 1 - r) * (1.0 - math.exp(-0.98 * N * p))
    return min(total, N)


def work(case):
    op = case["op"]
    if op in ("embed_fwd", "embed_bwd"):
        N, H, V = case["N"], case["H"], case["V"]
        e = 2 if case["dtype"] == "bf16" else 4
        if op == "embed_fwd":
            return {"bytes": 8 * N + e * H * (N + _unique(N, V)), "flops": N * H}
        out = 8 * _unique(N, V) * H if case["accumulate"] else 4 * V * H
        return {"bytes": 8 * N + e * N * H + out, "flops": 2 * N * H}
    if op in ("attn_fwd", "attn_train"):
        lens, Hq, Hkv, D = _lens(case), case["Hq"], case["Hkv"], case["D"]
        T = sum(lens)
        pairs = Hq * sum(n * (n + 1) / 2 for n in lens)
        io = 2 * T * D * (2 * Hq + 2 * Hkv) + 4 * T * Hq
        if op == "attn_fwd":
            return {"bytes": io, "flops": 4 * D * pairs}
        return {"bytes": io + 2 * T * D * (2 * Hq + 2 * Hkv), "flops": (4 + 10) * D * pairs}
    B, k, n = case["B"], min(case["m"], case["n"]), max(case["m"], case["n"])
    e = 2 if case["dtype"] == "bf16" else 4
    # X X^T and its square are symmetric: half of each is work
    return {"bytes": B * k * n * (e + 2), "flops": 5.0 * B * (k * k * n + k ** 3 + 2 * k * k * n)}


# ---------------------------------------------------- 64 bits, definitions
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        out = torch.zeros(case["N"], case["H"], dtype=torch.float64, device="cuda")
        keep = s["ids"] != IGN
        out[keep] = s["W"].double()[s["ids"][keep]] * case["scale"]
        return out
    if op == "embed_bwd":
        out = torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
        keep = s["ids"] != IGN
        out.index_add_(0, s["ids"][keep], s["dY"][keep].double())
        out *= case["scale"]
        if case["accumulate"]:
            out += s["dW"].double()
        return out
    if op == "orthogonalize":
        a, b, c = COEFFS
        out = []
        for G in s["G"].double():
            X = G / (torch.linalg.norm(G) + EPS)
            for _ in range(5):
                if G.shape[0] <= G.shape[1]:
                    M = X @ X.T
                    X = a * X + b * (M @ X) + c * (M @ (M @ X))
                else:
                    M = X.T @ X
                    X = a * X + b * (X @ M) + c * ((X @ M) @ M)
            out.append(X)
        return torch.stack(out)
    lens, Hq, Hkv, D = _lens(case), case["Hq"], case["Hkv"], case["D"]
    T = sum(lens) + case["pad"]
    z = dict(dtype=torch.float64, device="cuda")
    o, dq = torch.zeros(T, Hq, D, **z), torch.zeros(T, Hq, D, **z)
    dk, dv = torch.zeros(T, Hkv, D, **z), torch.zeros(T, Hkv, D, **z)
    lse = torch.full((Hq, T), -math.inf, **z)
    t0 = 0
    for n in lens:
        r = slice(t0, t0 + n)
        t0 += n
        if n == 0:
            continue
        hide = torch.ones(n, n, dtype=torch.bool, device="cuda").triu_(1)
        for h in range(Hq):
            j = h * Hkv // Hq
            q, k, v = s["q"][r, h].double(), s["k"][r, j].double(), s["v"][r, j].double()
            S = ((q @ k.T) / math.sqrt(D)).masked_fill_(hide, -math.inf)
            lse[h, r] = torch.logsumexp(S, 1)
            P = torch.exp(S - lse[h, r][:, None])
            o[r, h] = P @ v
            if op == "attn_train":
                d = s["dO"][r, h].double()
                dv[r, j] += P.T @ d
                dP = d @ v.T
                dS = P * (dP - (P * dP).sum(1, keepdim=True)) / math.sqrt(D)
                dq[r, h] = dS @ k
                dk[r, j] += dS.T @ q
    out = {"o": o, "lse": lse}
    if op == "attn_train":
        out.update(dq=dq, dk=dk, dv=dv)
    return out
