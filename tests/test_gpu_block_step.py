"""The operators between blocks together, as a model uses them: a transformer block with norms
on both sides, a gate, checkpointed projections, packed attention and the head, its gradients
against autograd in 64 bits and against differences; captured into a graph; second
derivatives, which are refused."""
import os
import subprocess
import sys

import pytest
import torch

import block_util as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
HEADS, KV, D = 4, 2, 64
HID = 256


def _params(seed, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def r(*s, std, mean=0.0):
        return (mean + std * torch.randn(s, generator=g, device=DEV)).to(dtype)

    return dict(embed=r(300, HID, std=0.5), n0=r(HID, std=0.1, mean=1.0),
                wqkv=r((HEADS + 2 * KV) * D, HID, std=HID ** -0.5),
                wo=r(HID, HEADS * D, std=HID ** -0.5), post=r(HID, std=0.1, mean=1.0),
                gate=r(HID, std=0.5), n1=r(HID, std=0.1, mean=1.0),
                up=r(512, HID, std=HID ** -0.5), down=r(HID, 512, std=512 ** -0.5),
                wg=r(HID, HID, std=HID ** -0.5), n2=r(HID, std=0.1, mean=1.0))


def _model(flce, p, ids, target, cu):
    """Loss of one block: x, z = join(embed); attention joined with norms before and after and
    a learned gate; a gated mlp joined with a gate computed for each element."""
    first = flce.ResidualNorm(checkpoint=True)
    join = flce.ResidualNorm(gate_act="tanh", checkpoint=True)
    last = flce.ResidualNorm(gate_act="sigmoid", beta=0.5)
    linear = flce.CheckpointedLinear()
    T = ids.shape[0]
    x, z, ck = first(flce.Embedding(scale=2.0)(p["embed"], ids), w_pre=p["n0"])
    q, k, v = linear(z, p["wqkv"], ck).view(T, -1, D).split([HEADS, KV, KV], 1)
    o = flce.PackedAttention()(q, k, v, cu).reshape(T, HEADS * D)
    x, z, ck = join(linear(o, p["wo"]), x, w_pre=p["n1"], w_post=p["post"], gate=p["gate"])
    y = linear(torch.relu(linear(z, p["up"], ck)), p["down"])
    x, z = last(y, x, w_pre=p["n2"], gate=linear(z, p["wg"], ck))
    return flce.LinearCrossEntropyLoss()(p["embed"], z, target)


def _reference(p, ids, target, cu):
    """The same in 64 bits, without checkpoints."""
    def rms(x, w):
        return x * (x.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * w

    T = ids.shape[0]
    x = p["embed"][ids] * 2.0
    z = rms(x, p["n0"])
    qkv = (z @ p["wqkv"].t()).view(T, -1, D)
    outs = []
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        q, k, v = (t.transpose(0, 1) for t in qkv[a:b].split([HEADS, KV, KV], 1))
        k, v = (t.repeat_interleave(HEADS // KV, 0) for t in (k, v))
        s = (q @ k.transpose(1, 2) * D ** -0.5).masked_fill(
            torch.ones(b - a, b - a, dtype=torch.bool, device=DEV).triu_(1), float("-inf"))
        outs.append((s.softmax(-1) @ v).transpose(0, 1).reshape(b - a, HEADS * D))
    x = x + torch.tanh(p["gate"]) * rms(torch.cat(outs) @ p["wo"].t(), p["post"])
    z = rms(x, p["n1"])
    y = torch.relu(z @ p["up"].t()) @ p["down"].t()
    x = x + 0.5 * torch.sigmoid(z @ p["wg"].t()) * y
    z = rms(x, p["n2"])
    return torch.nn.functional.cross_entropy(z @ p["embed"].t(), target, ignore_index=-100)


def _batch(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    lens = [70, 1, 200, 129]
    cu = torch.tensor([0, 70, 71, 271, 400], dtype=torch.int32, device=DEV)
    ids = torch.randint(0, 300, (sum(lens),), generator=g, device=DEV)
    target = torch.randint(0, 300, (sum(lens),), generator=g, device=DEV)
    target[::9] = -100
    return ids, target, cu


def test_gradients_of_a_block(cuda_lib):
    """Of each gradient's norm: the checkpoints' values are off by up to 2^-4 of themselves,
    on average (over a binade, evenly spread, uniform within a step of 1/16 to 1/8 of the
    value) by 2.7e-2 in square mean, each by itself, which reaches the gradients of the
    weights they multiply and no others.  bf16 makes 2^-9.3 per rounding, of which
    the longest way has about twenty: 8e-3, twice that for what a small difference amplifies.
    Together below 4e-2 for weights behind a checkpoint and 2e-2 for the rest.

    The gradient of `up` also passes through the relu's mask.  Six roundings on the way to its
    input (embedding, o, attention's output, the join, z, the product), 2^-9.8 of a value each
    in square mean, put the input's noise at r = 2.8e-3 of its spread; a normal value and the
    same with noise r differ in sign for r / pi of all elements.  Such an element's gradient is
    there instead of not, or the reverse; half of all are there, so the square error is
    2 r / pi of the gradient's square: sqrt(1.8e-3) = 4.2e-2, and with the 4e-2 above, which is
    independent of it, sqrt(4.2e-2^2 + 4e-2^2) = 5.8e-2."""
    import linear_cross_entropy_fwd_gb300 as flce
    ids, target, cu = _batch(1)
    p = {k: v.requires_grad_() for k, v in _params(0).items()}
    loss = _model(flce, p, ids, target, cu)
    loss.backward()
    q = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    want = _reference(q, ids, target, cu)
    want.backward()
    assert abs(loss.item() - want.item()) <= 1e-2 * want.item()
    for k, v in q.items():
        err = ((p[k].grad.double() - v.grad).norm() / v.grad.norm()).item()
        assert err <= (5.8e-2 if k == "up" else 4e-2 if k in ("wqkv", "wo", "down", "wg")
                       else 2e-2), (k, err)


def test_gradients_against_differences(cuda_lib):
    """Along a direction of fp32 parameters of one join, the loss in fp32 goes as its gradient
    says: central differences of h = 2^-7 are off by h^2 / 6 of third derivatives, and by
    rounding, 2^-24 of the sum of magnitudes over h."""
    import linear_cross_entropy_fwd_gb300 as flce
    N, H = 40, 328
    for kind, act in (("rms", "tanh"), ("layer", "sigmoid")):
        g = torch.Generator(device=DEV).manual_seed(4)

        def r(*s):
            return torch.randn(s, generator=g, device=DEV)

        p = dict(y=r(N, H), h=r(N, H), w_pre=r(H), w_post=r(H), b_pre=r(H), b_post=r(H),
                 gate=r(N, H))
        A, B = r(N, H), r(N, H)
        join = flce.ResidualNorm(kind, gate_act=act, alpha=0.8, beta=1.2)

        def f(t):
            t = dict(t)
            ho, z = join(t.pop("y"), t.pop("h"), **t)
            return (ho.double() * A).sum() + (z.double() * B).sum()

        leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
        f(leaves).backward()
        for k in p:
            d = r(*p[k].shape) / p[k].numel() ** 0.5
            slope = (leaves[k].grad.double() * d).sum().item()
            e = 2.0 ** -7
            up, down = (f({**p, k: p[k] + s * e * d}).item() for s in (1, -1))
            size = (leaves[k].grad.double() * d).norm().item()
            noise = 2.0 ** -24 * 8 * (A.abs().sum() + B.abs().sum()).item() ** 0.5 / e
            assert abs((up - down) / (2 * e) - slope) <= 1e-3 * size + noise, k


def test_captured_block(cuda_lib):
    """Forward and backward in a graph, replayed on other values: the bits of a step outside."""
    import linear_cross_entropy_fwd_gb300 as flce
    p = {k: v.requires_grad_() for k, v in _params(0).items()}
    ids, target, cu = _batch(1)
    leaves = list(p.values())

    def step():
        loss = _model(flce, p, ids, target, cu)
        return (loss.detach(), *torch.autograd.grad(loss, leaves))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (5, 6):
        with torch.no_grad():
            for k, v in _params(seed).items():
                p[k].copy_(v)
            for a, b in zip((ids, target), _batch(seed)):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for a, b in zip(got, step()):
            assert torch.equal(a, b) and bool(torch.isfinite(a.float()).all())


def test_modules_take_any_layout(cuda_lib):
    """Transposed and broadcast inputs and gradients, batch axes, a stream that is not used, and
    inputs without a gradient."""
    import linear_cross_entropy_fwd_gb300 as flce
    N, H = 24, 64
    y = torch.randn(H, N, device=DEV).t().requires_grad_()
    h = torch.randn(1, H, device=DEV).expand(N, H)
    gate = torch.randn(N, 1, device=DEV).expand(N, 1).requires_grad_()
    w = torch.randn(2 * H, device=DEV)[::2].requires_grad_()
    join = flce.ResidualNorm("layer", gate_act="sigmoid")
    ho, z = join(y, h, w_pre=w, gate=gate)
    ho.sum().backward()  # z is not used; the gradient is a broadcast scalar
    p = dict(w_pre=w.detach(), b_pre=None, w_post=None, b_post=None, gate=gate.detach())
    opts = dict(kind="layer", gate_act="sigmoid", alpha=1.0, beta=1.0, eps=1e-6,
                post_norm=False, pre_norm=True)
    want = ref.join_grads(torch.zeros(N, H, device=DEV), torch.ones(N, H, device=DEV), y.detach(),
                          ho.detach(), p, opts)
    ref.check(y.grad, *want["dy"], "dy")
    ref.check(gate.grad, *want["dgate"], "dgate")
    assert not w.grad.any()
    x = torch.randn(2, 3, 64, device=DEV).to(BF).requires_grad_()
    W = torch.randn(48, 64, device=DEV).to(BF).requires_grad_()
    out = flce.CheckpointedLinear()(x, W)
    assert out.shape == (2, 3, 48) and torch.equal(out, x @ W.t())
    out.sum().backward()
    stored = flce.flce_ckpt_load(flce.flce_ckpt_save(x.detach().view(6, 64))).double()
    assert torch.equal(W.grad, stored.sum(0).to(BF).expand(48, 64))
    only_w = flce.CheckpointedLinear()(x.detach(), W)
    dW, = torch.autograd.grad(only_w.sum(), W)
    assert torch.equal(dW, W.grad)


def test_second_derivatives_are_refused(cuda_lib):
    import linear_cross_entropy_fwd_gb300 as flce
    x = torch.randn(16, 64, device=DEV).to(BF).requires_grad_()
    W = torch.randn(64, 64, device=DEV).to(BF).requires_grad_()
    for f, leaf in ((lambda: flce.ResidualNorm()(x)[1], x),
                    (lambda: flce.CheckpointedLinear()(x, W), W)):
        y = f().float().pow(2).sum()
        g, = torch.autograd.grad(y, leaf, create_graph=True)
        with pytest.raises(RuntimeError):
            g.float().pow(2).sum().backward()


def test_other_streams(cuda_lib):
    """A chain of calls on a side stream, its scratch from the pool, beside another's."""
    flce = cuda_lib
    x = torch.randn(3000, 1024, device=DEV).to(BF)
    dY = torch.randn(3000, 512, device=DEV).to(BF)

    def chain():
        ck = flce.Checkpoint.empty(3000, 1024, DEV)
        _, z, _ = flce.flce_resnorm_fwd(x, x, checkpoint=ck)
        return z, flce.flce_ckpt_wgrad(dY, ck)

    want = chain()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(chain())
    torch.cuda.synchronize()
    for a in got:
        assert all(torch.equal(u, v) for u, v in zip(a, want))


FIRST = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import linear_cross_entropy_fwd_gb300 as flce
g = torch.Generator(device="cuda").manual_seed(1)
BF = torch.bfloat16
def r(*s):
    return torch.randn(*s, generator=g, device="cuda").to(BF)
N, H = 300, int(sys.argv[2])
y, h, dz, dh, w, b, gate = r(N, H), r(N, H), r(N, H), r(N, H), r(H), r(H), r(N, 1)
kw = dict(w_pre=w, w_post=w, b_post=b, gate=gate, gate_act="tanh", kind="layer")
def run():
    out, z, stats = flce.flce_resnorm_fwd(y, h, **kw)
    grads = flce.flce_resnorm_bwd(dz, dh, y, out, stats, **kw)
    ck = flce.flce_ckpt_save(z)
    dW = flce.flce_ckpt_wgrad(dz, ck)
    return [out, z, stats, *grads, ck.data, dW, flce.flce_ckpt_load(ck)]
# one call that takes scratch, for the device's state; none of the kernels below
flce.flce_embed_bwd(y[:8], torch.zeros(8, dtype=torch.int64, device="cuda"), 16)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
want = run()
torch.cuda.synchronize()
assert len(got) == len(want)
for i, (a, e) in enumerate(zip(got, want)):
    assert (a is None) == (e is None) and (a is None or torch.equal(a, e)), i
print("same")
"""


@pytest.mark.parametrize("H", [1000, 5000])
def test_first_calls_inside_a_capture(cuda_lib, H):
    """Kernels that nothing has warmed up: attributes and launch shapes are found in the capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST, root, str(H)], capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "same", p.stdout + p.stderr
