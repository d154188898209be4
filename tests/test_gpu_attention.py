"""Packed causal attention and its gradients against 64-bit formulas.

Tolerances, element by element, with u = 2^-8 (half a step of bf16) and
e = 2^-16 for everything done in fp32 (sums of up to 128 products, 2^x, the
products with the scale; each is a few 2^-22 of the terms' sizes):
  o    u |o| (stored) + (u + e) P |V|            (P rounded to bf16)
  lse  e (1 + |lse|)
  dv   u |dv| + (u + e) P^T |dO|
  dS   u |dS| + P (E_delta + e (|dO| |V|^T + |delta|)) + e |dS|, where
       E_delta = |dO| . E_o comes from the stored o
  dq   u |dq| + scale E_dS |K|,   dk   u |dk| + scale E_dS^T |Q|
Numbers below the types' normal range have steps of their own: P below 2^-126
may become 0, and a stored bf16 is off by half of its least step, 2^-134."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, E = 2.0 ** -8, 2.0 ** -16


def _inputs(lens, Hq, Hkv, D, seed, pad=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + pad
    qkv = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * std).bfloat16().to(DEV)
    dO = torch.randn(T, Hq, D, generator=g).bfloat16().to(DEV)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], dO, cu


def _reference(q, k, v, dO, lens, scale, first=0):
    """64-bit outputs and their tolerances, as (name -> (value, bound))."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    z = dict(dtype=torch.float64, device=q.device)
    val = {"o": torch.zeros(T, Hq, D, **z), "dq": torch.zeros(T, Hq, D, **z),
           "dk": torch.zeros(T, Hkv, D, **z), "dv": torch.zeros(T, Hkv, D, **z),
           "lse": torch.full((Hq, T), -math.inf, **z)}
    tol = {n: torch.zeros_like(t) for n, t in val.items()}
    t0 = first
    for n in lens:
        r = slice(t0, t0 + n)
        t0 += n
        if n == 0:
            continue
        hide = torch.ones(n, n, dtype=torch.bool, device=q.device).triu_(1)
        for h in range(Hq):
            j = h // (Hq // Hkv)
            Q, K, V, G = (x.double() for x in (q[r, h], k[r, j], v[r, j], dO[r, h]))
            S = (Q @ K.T * scale).masked_fill(hide, -math.inf)
            lse = torch.logsumexp(S, 1)
            P = torch.exp(S - lse[:, None])
            O = P @ V
            F = torch.full_like(P, 2.0 ** -126).masked_fill(hide, 0)  # what P may lose
            Eo = U * O.abs() + ((U + E) * P + F) @ V.abs()
            dP = G @ V.T
            delta = (G * O).sum(1, keepdim=True)
            dS = P * (dP - delta)
            Ed = (G.abs() * Eo).sum(1, keepdim=True)
            size = G.abs() @ V.abs().T + delta.abs()
            EdS = (U + E) * dS.abs() + P * (Ed + E * size) + F * size
            val["o"][r, h], tol["o"][r, h] = O, Eo
            val["lse"][h, r], tol["lse"][h, r] = lse, E * (1 + lse.abs())
            dq = dS @ K * scale
            val["dq"][r, h], tol["dq"][r, h] = dq, U * dq.abs() + scale * (EdS @ K.abs())
            val["dk"][r, j] += dS.T @ Q * scale
            tol["dk"][r, j] += scale * (EdS.T @ Q.abs())
            val["dv"][r, j] += P.T @ G
            tol["dv"][r, j] += ((U + E) * P + F).T @ G.abs()
    for n in ("dk", "dv"):
        tol[n] += U * val[n].abs()
    for n in ("o", "dq", "dk", "dv"):
        tol[n] += 2.0 ** -134
    return val, tol


def _close(name, got, val, tol):
    got = got.double()
    same = got == val  # equal infinities too
    err = torch.where(same, 0.0, (got - val).abs())
    worst = (err - tol).max().item() if got.numel() else 0.0
    assert bool(((err <= tol) | same).all()), f"{name}: {worst:.3g} over its bound"


def _run(lib, q, k, v, dO, cu, **kw):
    o, lse = lib.flce_attn_fwd(q, k, v, cu, sync=True, **kw)
    dq, dk, dv = lib.flce_attn_bwd(dO, q, k, v, o, lse, cu, sync=True, **kw)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


@pytest.mark.parametrize("lens,Hq,Hkv,D,pad", [
    ([1], 1, 1, 64, 0),
    ([2], 1, 1, 128, 0),
    ([128], 2, 1, 128, 0),
    ([129], 2, 2, 64, 3),
    ([256], 1, 1, 128, 0),
    ([127, 128, 0, 1, 300], 4, 2, 128, 5),
    ([0, 0, 70, 0], 4, 1, 64, 0),
    ([5] * 40, 2, 1, 64, 1),
    ([640], 8, 2, 128, 0),
    ([1000, 37], 6, 3, 64, 0),
    ([300, 201], 3, 1, 80, 2),      # head sizes between the kernels' 64 and 128
    ([150, 10], 2, 1, 8, 0),
    ([200], 2, 2, 120, 0),
    ([65, 66], 2, 1, 40, 0),
])
def test_attention(cuda_lib, lens, Hq, Hkv, D, pad):
    q, k, v, dO, cu = _inputs(lens, Hq, Hkv, D, sum(lens) + D, pad)
    got = _run(cuda_lib, q, k, v, dO, cu)
    val, tol = _reference(q, k, v, dO, lens, D ** -0.5)
    for n in val:
        _close(n, got[n], val[n], tol[n])
    again = _run(cuda_lib, q, k, v, dO, cu)
    for n in val:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("scale,std", [(0.02, 1.0), (1.0, 3.0), (2.0, 4.0)])
def test_attention_scales(cuda_lib, scale, std):
    """Scores from nearly flat to several hundred apart, so that the running
    maximum moves often and most of P vanishes."""
    lens = [500, 140]
    q, k, v, dO, cu = _inputs(lens, 2, 1, 64, 7, std=std)
    got = _run(cuda_lib, q, k, v, dO, cu, scale=scale)
    val, tol = _reference(q, k, v, dO, lens, scale)
    # scores of size s lose s 2^-24 each in fp32, and P = exp(S - lse) as much relative to itself
    big = (q.double().norm(dim=2).max() * k.double().norm(dim=2).max() * scale).item()
    extra = 8 * big * 2.0 ** -24
    for n in val:
        grow = (1 + extra / E) if n == "lse" else (1 + extra / U) * (1 + extra / E)
        _close(n, got[n], val[n], tol[n] * grow)


def test_attention_rising_scores(cuda_lib):
    """Every key tile raises the maximum by more than the rescaling threshold."""
    T, D = 700, 64
    q = torch.ones(T, 1, D, device=DEV).bfloat16()
    k = (torch.arange(T, device=DEV) / 16.0)[:, None, None].expand(T, 1, D).bfloat16().contiguous()
    v = torch.randn(T, 1, D, device=DEV).bfloat16()
    dO = torch.randn(T, 1, D, device=DEV).bfloat16()
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    got = _run(cuda_lib, q, k, v, dO, cu, scale=1.0 / 16)
    val, tol = _reference(q, k, v, dO, [T], 1.0 / 16)
    for n in val:
        _close(n, got[n], val[n], tol[n] * 2)  # scores up to 175: 175 2^-24 beside e


def test_attention_strides(cuda_lib):
    """Separate head-major tensors, gradients into slices of one buffer."""
    lens, Hq, Hkv, D = [200, 77], 4, 2, 64
    q, k, v, dO, cu = _inputs(lens, Hq, Hkv, D, 3)
    ref = _run(cuda_lib, q, k, v, dO, cu)
    T = q.shape[0]

    def head_major(x):
        return x.transpose(0, 1).contiguous().transpose(0, 1)

    q2, k2, v2, dO2 = (head_major(x) for x in (q, k, v, dO))
    out = torch.empty(T, Hq, 2 * D, device=DEV, dtype=torch.bfloat16)[:, :, D:]
    o, lse = cuda_lib.flce_attn_fwd(q2, k2, v2, cu, out=out)
    assert o.data_ptr() == out.data_ptr()
    buf = torch.empty(T, Hq + 2 * Hkv, D, device=DEV, dtype=torch.bfloat16)
    cuda_lib.flce_attn_bwd(dO2, q2, k2, v2, o, lse, cu, dq=buf[:, :Hq], dk=buf[:, Hq:Hq + Hkv],
                           dv=buf[:, Hq + Hkv:])
    assert torch.equal(o, ref["o"]) and torch.equal(lse, ref["lse"])
    assert torch.equal(buf, torch.cat([ref["dq"], ref["dk"], ref["dv"]], 1))


def test_attention_other_sequences_values_stay_out(cuda_lib):
    """NaN and infinities in a neighbouring sequence, and in tokens of no sequence,
    change no bit of the others."""
    lens = [100, 130, 50]
    q, k, v, dO, cu = _inputs(lens, 2, 1, 64, 11, pad=9)
    cu = cu + 4  # four tokens before the first sequence, five after the last
    ref = _run(cuda_lib, q, k, v, dO, cu)
    bad = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)
    bad[:4] = bad[284:] = bad[104:234] = True
    q2, k2, v2, dO2 = (x.clone() for x in (q, k, v, dO))
    for i, x in enumerate((q2, k2, v2, dO2)):
        x[bad] = [float("nan"), float("inf"), -float("inf"), float("nan")][i]
    got = _run(cuda_lib, q2, k2, v2, dO2, cu)
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[n][~bad], ref[n][~bad]), n
        outside = torch.cat([got[n][:4], got[n][284:]])
        assert not outside.any(), n
    assert torch.equal(got["lse"][:, ~bad], ref["lse"][:, ~bad])
    assert bool((got["lse"][:, :4] == -math.inf).all() and (got["lse"][:, 284:] == -math.inf).all())


def test_attention_no_sequences(cuda_lib):
    q, k, v, dO, _ = _inputs([10], 2, 1, 64, 1)
    for cu in ([0], [3], [7, 7, 7]):
        got = _run(cuda_lib, q, k, v, dO, torch.tensor(cu, dtype=torch.int32, device=DEV))
        for n in ("o", "dq", "dk", "dv"):
            assert not got[n].any()
        assert bool((got["lse"] == -math.inf).all())
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    got = _run(cuda_lib, e, e[:, :1], e[:, 1:], e, cu)
    assert got["o"].shape == (0, 2, 64) and got["lse"].shape == (2, 0)


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [-1, 50, 100], [0, 101], [2 ** 31 - 1, 5]])
def test_attention_bad_offsets(cuda_lib, cu):
    """Offsets out of order or out of range: an error, zeros, nothing read or written astray."""
    q, k, v, dO, _ = _inputs([100], 2, 1, 64, 2)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    info = {}
    o, lse = cuda_lib.flce_attn_fwd(q, k, v, cu, info=info)
    assert int(info["status"].item()) == cuda_lib.FLCE_ERR_ARG
    assert not o.any() and bool((lse == -math.inf).all())
    with pytest.raises(cuda_lib.FlceError) as e:
        cuda_lib.flce_attn_bwd(dO, q, k, v, o, lse, cu, sync=True)
    assert e.value.status == cuda_lib.FLCE_ERR_ARG


def test_attention_refusals(cuda_lib):
    q, k, v, dO, cu = _inputs([64], 4, 2, 64, 4)
    o, lse = cuda_lib.flce_attn_fwd(q, k, v, cu)
    for kw in (dict(q=q.float()), dict(k=k[:32]), dict(q=q.cpu()), dict(cu=cu.long()),
               dict(v=v.transpose(1, 2)), dict(q=q[:, :3])):
        a = dict(q=q, k=k, v=v, cu=cu)
        a.update(kw)
        with pytest.raises((ValueError, TypeError, cuda_lib.FlceError)):
            cuda_lib.flce_attn_fwd(a["q"], a["k"], a["v"], a["cu"])
    with pytest.raises(cuda_lib.FlceError):  # broadcast heads have stride 0
        cuda_lib.flce_attn_fwd(q, k[:, :1].expand(-1, 2, -1), v, cu)
    with pytest.raises(cuda_lib.FlceError) as e:  # 8 bytes off a 16-byte boundary
        cuda_lib.flce_attn_fwd(torch.empty(64 * 256 + 4, dtype=torch.bfloat16, device=DEV)[4:]
                               .view(64, 4, 64), k, v, cu)
    assert e.value.status == cuda_lib.FLCE_ERR_ALIGN
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(cuda_lib.FlceError):
            cuda_lib.flce_attn_fwd(q, k, v, cu, scale=scale)
    with pytest.raises(ValueError):
        cuda_lib.flce_attn_bwd(dO, q, k, v, o, lse[:2], cu)


def test_attention_side_stream_and_workspace(cuda_lib):
    q, k, v, dO, cu = _inputs([400, 90], 4, 2, 128, 5)
    ref = _run(cuda_lib, q, k, v, dO, cu)
    info = {}
    cuda_lib.flce_attn_bwd(dO, q, k, v, ref["o"], ref["lse"], cu, info=info)
    ws = torch.empty(info["workspace_bytes"], dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = cuda_lib.flce_attn_fwd(q, k, v, cu, workspace=ws)
        dq, dk, dv = cuda_lib.flce_attn_bwd(dO, q, k, v, o, lse, cu, workspace=ws)
    side.synchronize()
    for n, x in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(x, ref[n]), n
    with pytest.raises(cuda_lib.FlceError) as e:
        cuda_lib.flce_attn_bwd(dO, q, k, v, o, lse, cu, workspace=ws[:-256])
    assert e.value.status == cuda_lib.FLCE_ERR_WORKSPACE


def test_attention_in_a_graph(cuda_lib):
    """Captured once, replayed on other values and other offsets."""
    q, k, v, dO, cu = _inputs([300, 40, 60], 4, 2, 64, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # per-device setup outside the capture
        o, lse = cuda_lib.flce_attn_fwd(q, k, v, cu)
        cuda_lib.flce_attn_bwd(dO, q, k, v, o, lse, cu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = cuda_lib.flce_attn_fwd(q, k, v, cu)
        dq, dk, dv = cuda_lib.flce_attn_bwd(dO, q, k, v, o, lse, cu)
    for lens in ([100, 0, 290], [1, 398, 1]):
        q2, k2, v2, dO2, cu2 = _inputs(lens, 4, 2, 64, sum(lens) + lens[0], pad=400 - sum(lens))
        for dst, src in ((q, q2), (k, k2), (v, v2), (dO, dO2), (cu, cu2)):
            dst.copy_(src)
        graph.replay()
        ref = _run(cuda_lib, q, k, v, dO, cu)
        for n, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
            assert torch.equal(x, ref[n]), n


def test_attention_gradient_by_differences(cuda_lib):
    """f = <C, o> along a direction, by differences of the 64-bit formula at both
    ends, against the module's gradients: the gradient is off by its tolerances'
    sum along the direction, and the difference by its third derivative."""
    lens, Hq, Hkv, D = [70, 131], 4, 2, 64
    q, k, v, C, cu = _inputs(lens, Hq, Hkv, D, 8)
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    o = cuda_lib.PackedAttention()(*x, cu)
    o.backward(C)
    _, tol = _reference(q, k, v, C, lens, D ** -0.5)
    for i, name in enumerate(("dq", "dk", "dv")):
        direction = torch.randn(x[i].shape, device=DEV, dtype=torch.float64)

        def f(step):
            y = [t.double() for t in (q, k, v)]
            y[i] = y[i] + step * direction
            val, _ = _reference(*y, C, lens, D ** -0.5)
            return (val["o"] * C.double()).sum()

        slope = ((f(1e-4) - f(-1e-4)) / 2e-4).item()
        got = (x[i].grad.double() * direction).sum().item()
        bound = (tol[name] * direction.abs()).sum().item()
        assert abs(got - slope) <= bound + 1e-5 * abs(slope), (name, got, slope, bound)
        # the errors have no common sign: far less than the worst case
        assert abs(got - slope) <= 0.1 * bound + 1e-5 * abs(slope), (name, got, slope, bound)


def test_attention_broadcast_heads_gradient(cuda_lib):
    """One k head expanded over two: its gradient is the sum over both."""
    q, k, v, C, cu = _inputs([90], 4, 2, 64, 9)
    k1 = k[:, :1].clone().requires_grad_()
    o = cuda_lib.PackedAttention()(q, k1.expand(-1, 2, -1), v, cu)
    o.backward(C)
    k2 = k1.detach().expand(-1, 2, -1).contiguous()
    o2, lse = cuda_lib.flce_attn_fwd(q, k2, v, cu)
    _, dk, _ = cuda_lib.flce_attn_bwd(C, q, k2, v, o2, lse, cu)
    assert torch.equal(o, o2)
    assert torch.equal(k1.grad, dk.sum(1, keepdim=True))


@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    ([900, 257, 0, 130, 4, 1100], 40, 8, 128),   # several units per CTA, with and without a second tile
    ([128] * 30 + [129] * 11, 16, 16, 64),
])
def test_attention_many_units(cuda_lib, lens, Hq, Hkv, D):
    """More units of work than the GPU has SMs."""
    q, k, v, dO, cu = _inputs(lens, Hq, Hkv, D, D, pad=3)
    got = _run(cuda_lib, q, k, v, dO, cu)
    val, tol = _reference(q, k, v, dO, lens, D ** -0.5)
    for n in val:
        _close(n, got[n], val[n], tol[n])


@pytest.mark.parametrize("lens,first,pad", [
    ([7], 0, 0),
    ([0, 40, 1, 0, 300, 0], 9, 3),      # tokens before the first sequence and after the last
    ([1] * 70, 1, 0),                   # more sequences than two warps have threads
    ([0, 0], 0, 50),                    # nothing but tokens outside
])
@pytest.mark.parametrize("status", [False, True])
def test_attention_few_units(cuda_lib, lens, first, pad, status):
    """A batch small enough to run without a plan gives what the same sequences give
    as the first ones of a batch that is not, bit for bit."""
    Hq, Hkv, D = 2, 1, 64
    q, k, v, _, cu = _inputs([first] + lens, Hq, Hkv, D, sum(lens), pad)
    cu = cu[1:].contiguous()
    T, B = q.shape[0], len(lens)
    o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Hq, T), 7.0, device=DEV)
    info = {} if status else None
    cuda_lib.flce_attn_fwd(q, k, v, cu, out=o, lse=lse, info=info)
    if status:
        assert int(info["status"].item()) == 0
    more = torch.cat([cu, cu[-1:].expand(400)])  # empty sequences: too many units for one round
    o2, lse2 = cuda_lib.flce_attn_fwd(q, k, v, more.contiguous())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    outside = torch.ones(T, dtype=torch.bool, device=DEV)
    outside[int(cu[0]):int(cu[-1])] = False
    assert not o[outside].any() and bool((lse[:, outside] == -math.inf).all())
    assert bool(torch.isfinite(lse[:, ~outside]).all())


@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    ([300, 90], 2, 1, 64),              # no plan
    ([300, 90], 4, 2, 128),
    ([290] + [40] * 60, 8, 2, 128),     # with one
])
def test_attention_bits_do_not_depend_on_what_follows(cuda_lib, lens, Hq, Hkv, D):
    """Queries of another sequence, of padding, or later in the same sequence share a
    block of rows with a token, and change no bit of its results."""
    q, k, v, dO, cu = _inputs(lens, Hq, Hkv, D, 21, pad=7)
    n = lens[0]
    ref = _run(cuda_lib, q, k, v, dO, cu)
    q2 = q.clone()
    q2[n:] *= 64.0      # finite, and enough to raise the maximum at every key tile
    got = _run(cuda_lib, q2, k, v, dO, cu)
    for name in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[name][:n], ref[name][:n]), name
    assert torch.equal(got["lse"][:, :n], ref["lse"][:, :n])
    q3 = q.clone()
    q3[n - 5:n] *= 64.0
    got = _run(cuda_lib, q3, k, v, dO, cu)
    for name in ("o", "dq"):
        assert torch.equal(got[name][:n - 5], ref[name][:n - 5]), name
    assert torch.equal(got["lse"][:, :n - 5], ref["lse"][:, :n - 5])


POISON = [("nan", float("nan")), ("inf", float("inf")), ("-inf", -float("inf"))]
POISONED_BATCHES = [
    # lengths, heads, head size, the poisoned sequence and token
    ([200, 300], 4, 2, 64, 1, 150),             # no plan; heads of a group shared out
    ([200, 300], 4, 2, 128, 1, 270),            # in the partial last tile
    ([300, 10], 2, 2, 80, 0, 100),              # first tile; its queries' pair reads it too
    ([100] * 45 + [700], 8, 8, 128, 45, 129),   # a plan
    ([60] * 30 + [513], 6, 3, 64, 30, 511),
]


def _poisoned(lens, Hq, Hkv, D, s, t, seed):
    q, k, v, dO, cu = _inputs(lens, Hq, Hkv, D, seed, pad=2)
    return q, k, v, dO, cu, int(cu[s]), int(cu[s]) + t, int(cu[s + 1])


@pytest.mark.parametrize("what,x", POISON)
@pytest.mark.parametrize("lens,Hq,Hkv,D,s,t", POISONED_BATCHES)
def test_attention_nonfinite_v(cuda_lib, lens, Hq, Hkv, D, s, t, what, x):
    """An element of one token's v reaches that column of o, from that token on."""
    q, k, v, dO, cu, a, i, b = _poisoned(lens, Hq, Hkv, D, s, t, 31)
    group, d, h = Hq // Hkv, D // 2 + 3, Hkv - 1
    o, lse = cuda_lib.flce_attn_fwd(q, k, v, cu)
    v2 = v.clone()
    v2[i, h, d] = x
    o2, lse2 = cuda_lib.flce_attn_fwd(q, k, v2, cu, sync=True)
    assert torch.equal(lse2, lse)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[i:b, h * group:(h + 1) * group, d] = True
    assert torch.equal(o2[~hit], o[~hit])
    want = torch.full((), x, dtype=o.dtype, device=DEV).expand(int(hit.sum()))
    assert torch.equal(o2[hit].nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


@pytest.mark.parametrize("what,x", POISON)
@pytest.mark.parametrize("lens,Hq,Hkv,D,s,t", POISONED_BATCHES)
def test_attention_nonfinite_k(cuda_lib, lens, Hq, Hkv, D, s, t, what, x):
    """A token's k reaches the outputs and dq of no token before it."""
    q, k, v, dO, cu, a, i, b = _poisoned(lens, Hq, Hkv, D, s, t, 32)
    group, h = Hq // Hkv, Hkv - 1
    ref = _run(cuda_lib, q, k, v, dO, cu)
    k2 = k.clone()
    k2[i, h, 5] = x
    got = _run(cuda_lib, q, k2, v, dO, cu)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[i:b, h * group:(h + 1) * group] = True
    assert torch.equal(got["o"][~hit], ref["o"][~hit])
    assert torch.equal(got["lse"].T[~hit], ref["lse"].T[~hit])
    assert torch.equal(got["dq"][~hit], ref["dq"][~hit])
    if what == "nan":
        assert bool(got["o"][hit].isnan().all() and got["dq"][hit].isnan().all())
    else:  # a score of -inf leaves o finite, and dq in that column 0 times infinity
        assert not bool(got["dq"][hit][:, 5].isfinite().any())
    hit = torch.zeros(k.shape[:2], dtype=torch.bool, device=DEV)
    hit[a:b, h] = True
    for n in ("dk", "dv"):
        assert torch.equal(got[n][~hit], ref[n][~hit]), n
        if what == "nan":
            assert bool(got[n][hit].isnan().all()), n


@pytest.mark.parametrize("what,x", POISON)
@pytest.mark.parametrize("lens,Hq,Hkv,D,s,t", POISONED_BATCHES)
def test_attention_nonfinite_q(cuda_lib, lens, Hq, Hkv, D, s, t, what, x):
    """One head's q of one token reaches its own o and dq, and dk and dv of the tokens
    that it sees: none after it."""
    q, k, v, dO, cu, a, i, b = _poisoned(lens, Hq, Hkv, D, s, t, 33)
    h = Hq - 1
    kvh = h // (Hq // Hkv)
    ref = _run(cuda_lib, q, k, v, dO, cu)
    q2 = q.clone()
    q2[i, h, 5] = x
    got = _run(cuda_lib, q2, k, v, dO, cu)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[i, h] = True
    for n in ("o", "dq"):
        assert torch.equal(got[n][~hit], ref[n][~hit]), n
        assert bool(got[n][hit].isnan().all()), n
    assert torch.equal(got["lse"].T[~hit], ref["lse"].T[~hit])
    hit = torch.zeros(k.shape[:2], dtype=torch.bool, device=DEV)
    hit[a:i + 1, kvh] = True
    for n in ("dk", "dv"):
        assert torch.equal(got[n][~hit], ref[n][~hit]), n
        assert bool(got[n][hit].isnan().all()), n


@pytest.mark.parametrize("what,x", POISON)
@pytest.mark.parametrize("lens,Hq,Hkv,D,s,t", POISONED_BATCHES)
def test_attention_nonfinite_dO(cuda_lib, lens, Hq, Hkv, D, s, t, what, x):
    """An element of one head's dO of one token reaches its own dq, dk of the tokens it
    sees, and that column of their dv: none after it."""
    q, k, v, dO, cu, a, i, b = _poisoned(lens, Hq, Hkv, D, s, t, 34)
    h, d = 0, D // 2 + 1
    ref = _run(cuda_lib, q, k, v, dO, cu)
    dO2 = dO.clone()
    dO2[i, h, d] = x
    got = _run(cuda_lib, q, k, v, dO2, cu)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[i, h] = True
    assert torch.equal(got["dq"][~hit], ref["dq"][~hit])
    assert not bool(got["dq"][hit].isfinite().any())
    hit = torch.zeros(k.shape[:2], dtype=torch.bool, device=DEV)
    hit[a:i + 1, 0] = True
    assert torch.equal(got["dk"][~hit], ref["dk"][~hit])
    assert not bool(got["dk"][hit].isfinite().any())
    hit = torch.zeros_like(k, dtype=torch.bool)
    hit[a:i + 1, 0, d] = True
    assert torch.equal(got["dv"][~hit], ref["dv"][~hit])
    assert not bool(got["dv"][hit].isfinite().any())


@pytest.mark.parametrize("D", [64, 128])
def test_attention_scores_of_minus_infinity(cuda_lib, D):
    """Keys that score -inf count for nothing, also where they fill the first key tile;
    a row that sees no others has an lse of -inf and no o."""
    lens, cut = [300, 40], 140
    q, k, v, dO, cu = _inputs(lens, 2, 1, D, 35)
    q, k = q.clone(), k.clone()
    q[..., 0] = q[..., 0].abs() + 0.5
    k[:cut, :, 0] = -math.inf
    o, lse = cuda_lib.flce_attn_fwd(q, k, v, cu, sync=True)
    val, tol = _reference(q, k, v, dO, lens, D ** -0.5)
    seen = slice(cut, sum(lens))
    _close("o", o[seen], val["o"][seen], tol["o"][seen])
    _close("lse", lse[:, seen], val["lse"][:, seen], tol["lse"][:, seen])
    assert bool((lse[:, :cut] == -math.inf).all() and o[:cut].isnan().all())


def test_attention_interleaved_and_in_place(cuda_lib):
    """q, k and v by turns within each head, gradients likewise, or over o; outputs over
    what is still read are refused."""
    T, H, D = 330, 3, 64
    lens = [200, 130]
    q, k, v, dO, cu = _inputs(lens, H, H, D, 36)
    ref = _run(cuda_lib, q, k, v, dO, cu)
    buf = torch.stack([q, k, v], 2).contiguous()          # [T, H, 3, D]
    a, b, c = buf.unbind(2)
    o, lse = cuda_lib.flce_attn_fwd(a, b, c, cu)
    grads = torch.empty_like(buf)
    cuda_lib.flce_attn_bwd(dO, a, b, c, o, lse, cu, dq=grads[:, :, 0], dk=grads[:, :, 1],
                           dv=grads[:, :, 2])
    assert torch.equal(o, ref["o"]) and torch.equal(lse, ref["lse"])
    for i, n in enumerate(("dq", "dk", "dv")):
        assert torch.equal(grads[:, :, i], ref[n]), n
    for n in ("dq", "dk", "dv"):
        over = o.clone()
        got = dict(zip(("dq", "dk", "dv"),
                       cuda_lib.flce_attn_bwd(dO, q, k, v, over, lse, cu, **{n: over})))
        for m in got:
            assert torch.equal(got[m], ref[m]), (n, m)
    for kw in (dict(out=a), dict(out=b)):
        with pytest.raises(cuda_lib.FlceError, match="overlaps"):
            cuda_lib.flce_attn_fwd(a, b, c, cu, **kw)
    for kw in (dict(dq=a), dict(dk=b), dict(dv=c), dict(dq=dO), dict(dk=grads[:, :, 0], dq=grads[:, :, 0])):
        with pytest.raises(cuda_lib.FlceError, match="overlaps"):
            cuda_lib.flce_attn_bwd(dO, a, b, c, o, lse, cu, **kw)


@pytest.mark.parametrize("cu,good", [([0], True), ([0, 0, 0], True), ([0, 5], False), ([-1, 0], False),
                                     ([2], False)])
def test_attention_offsets_without_tokens(cuda_lib, cu, good):
    """No token, but offsets: they are checked all the same."""
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 0, device=DEV)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    info = {}
    want = cuda_lib.FLCE_OK if good else cuda_lib.FLCE_ERR_ARG
    cuda_lib.flce_attn_fwd(e, e, e, cu, info=info)
    assert int(info["status"].item()) == want
    cuda_lib.flce_attn_bwd(e, e, e, e, e, lse, cu, info=info)
    assert int(info["status"].item()) == want
    cuda_lib.flce_attn_fwd(e, e, e, cu)          # nobody looks: nothing to do
    if not good:
        with pytest.raises(cuda_lib.FlceError):
            cuda_lib.flce_attn_bwd(e, e, e, e, e, lse, cu, sync=True)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([4500], 2, 1, 128), ([3001, 1700], 2, 1, 64),
                                           ([2600, 77], 3, 1, 80)])
def test_attention_long_sequences(cuda_lib, lens, Hq, Hkv, D):
    """Dozens of key tiles per row.  fp32 sums of n terms in chains of 32 per tile, then
    over the tiles: (32 + n / 128) 2^-24 of the terms' sizes, within e up to 28,000."""
    q, k, v, dO, cu = _inputs(lens, Hq, Hkv, D, D + 1, pad=5)
    got = _run(cuda_lib, q, k, v, dO, cu)
    val, tol = _reference(q, k, v, dO, lens, D ** -0.5)
    for n in val:
        _close(n, got[n], val[n], tol[n])
