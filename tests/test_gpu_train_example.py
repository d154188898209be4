"""The operators together, as examples/train_tied_lm.py uses them: its gradients
against autograd in 64 bits, and a loss that falls."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def _reference_grads(model, ids, target, cu):
    E, Wqkv, Wo = (getattr(model, n).bfloat16().double().requires_grad_()
                   for n in ("embed", "wqkv", "wo"))
    Hq, Hkv, D, T = model.heads_q, model.heads_kv, model.dim, ids.shape[0]
    x = E[ids] * model.scale
    qkv = (x @ Wqkv).view(T, Hq + 2 * Hkv, D)
    out = []
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        q, k, v = (t.transpose(0, 1) for t in (qkv[a:b, :Hq], qkv[a:b, Hq:Hq + Hkv],
                                               qkv[a:b, Hq + Hkv:]))
        k, v = (t.repeat_interleave(Hq // Hkv, 0) for t in (k, v))
        s = (q @ k.transpose(1, 2) * D ** -0.5).masked_fill(
            torch.ones(b - a, b - a, dtype=torch.bool, device=ids.device).triu_(1), float("-inf"))
        out.append((s.softmax(-1) @ v).transpose(0, 1).reshape(b - a, Hq * D))
    y = x + torch.cat(out) @ Wo
    loss = torch.nn.functional.cross_entropy(y @ E.T, target, ignore_index=-100)
    loss.backward()
    return loss.item(), {"embed": E.grad, "wqkv": Wqkv.grad, "wo": Wo.grad}


def test_gradients_of_the_whole_step(cuda_lib):
    """bf16 activations and gradients: each of the eight roundings on the longest
    way (x, qkv, P, o, y, G, dy, dS, ...) is at most 2^-8 of a value and about
    2^-9.3 on average; eight independent ones make 4.5e-3 of a gradient's norm,
    and 2e-2 leaves room for those that a small difference amplifies."""
    import train_tied_lm as ex
    model = ex.TiedLM(vocab=512, hidden=256, heads_q=4, heads_kv=2)
    ids, target, cu = ex.batch(512, [70, 1, 200, 129], 3)
    loss, grads = model.loss_and_grads(ids, target, cu)
    ref_loss, ref = _reference_grads(model, ids, target, cu)
    assert abs(loss.item() - ref_loss) <= 1e-2 * abs(ref_loss)
    for n, g in ref.items():
        err = (grads[n].double() - g).norm() / g.norm()
        assert err.item() <= 2e-2, (n, err.item())


def test_loss_falls(cuda_lib):
    import train_tied_lm as ex
    losses = ex.train(steps=40)
    assert all(x == x for x in losses)
    # from about ln 4096 = 8.3 at the start
    assert losses[0] > 7.0 and losses[-1] < 0.6 * losses[0], losses
