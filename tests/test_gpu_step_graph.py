"""A training step through the modules, captured into a CUDA graph: embedding,
attention, their gradients, and the orthogonalised update.  And second
derivatives, which they refuse."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _step(flce, E, Wqkv, ids, cu, C, heads, D):
    Hq, Hkv = heads
    x = flce.Embedding(scale=2.0)(E, ids)
    q, k, v = (x @ Wqkv).view(ids.shape[0], Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)
    o = flce.PackedAttention()(q, k, v, cu)
    dE, dW = torch.autograd.grad([o], [E, Wqkv], [C])
    return o.detach(), dE, dW, flce.flce_orthogonalize(dW)


def test_captured_training_step(cuda_lib):
    """Replayed on other values, it gives what a step outside a graph gives, bit
    for bit: no kernel's result depends on timing."""
    import linear_cross_entropy_fwd_gb300 as flce
    T, H, V, heads, D = 300, 128, 500, (4, 2), 64
    g = torch.Generator(device="cuda").manual_seed(5)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    E = randn(V, H).requires_grad_()
    Wqkv = (randn(H, (heads[0] + 2 * heads[1]) * D) * 0.1).requires_grad_()
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    cu = torch.tensor([0, 40, 41, 41, 290], dtype=torch.int32, device="cuda")
    C = randn(T, heads[0], D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # per-device setup outside the capture; its graph is dropped
        _step(flce, E, Wqkv, ids, cu, C, heads, D)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _step(flce, E, Wqkv, ids, cu, C, heads, D)
    for cuts in ([0, 300, 300, 300, 300], [0, 1, 130, 257, 299]):
        with torch.no_grad():
            E.copy_(randn(V, H))
            ids.copy_(torch.randint(0, V, (T,), generator=g, device="cuda"))
            cu.copy_(torch.tensor(cuts, dtype=torch.int32))
            C.copy_(randn(T, heads[0], D))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for a, b in zip(got, _step(flce, E, Wqkv, ids, cu, C, heads, D)):
            assert torch.equal(a, b)
            assert torch.isfinite(a.float()).all() and a.float().abs().sum() > 0


def test_second_derivatives_are_refused(cuda_lib):
    import linear_cross_entropy_fwd_gb300 as flce
    E = torch.randn(20, 64, device="cuda").bfloat16().requires_grad_()
    ids = torch.arange(10, device="cuda")
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    for f in (lambda: flce.Embedding()(E, ids),
              lambda: flce.PackedAttention()(*(E[:10].view(10, 1, 64),) * 3, cu)):
        y = f().float().pow(2).sum()
        g, = torch.autograd.grad(y, E, create_graph=True)
        with pytest.raises(RuntimeError):
            g.float().pow(2).sum().backward()
