"""Bounds of the operators around the head.  Every buffer they write lies in the
middle of a larger one whose other bytes hold a pattern that has to survive; the
outputs themselves start as NaN and have to be written whole.  And addresses
beyond 2^31 elements from a buffer's start."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAND = 4096  # bytes on each side


class Guarded:
    def __init__(self, shape, dtype, fill=float("nan")):
        n = torch.empty(0, dtype=dtype).element_size()
        for s in shape:
            n *= s
        self.n = n
        self.raw = torch.full((n + 2 * BAND,), 0x5A, dtype=torch.uint8, device=DEV)
        self.t = self.raw[BAND:BAND + n].view(dtype).view(shape)
        if dtype.is_floating_point:
            self.t.fill_(fill)

    def check(self, name, whole=True):
        assert bool((self.raw[:BAND] == 0x5A).all()), f"{name}: bytes before it"
        assert bool((self.raw[BAND + self.n:] == 0x5A).all()), f"{name}: bytes after it"
        if whole and self.t.dtype.is_floating_point:
            assert not bool(self.t.isnan().any()), f"{name}: not written whole"


@pytest.mark.parametrize("N,H,V", [(1, 8, 1), (33, 136, 77), (2100, 1000, 301), (5000, 64, 40000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_embed_bounds(cuda_lib, N, H, V, dtype):
    W = torch.randn(V, H, device=DEV).to(dtype)
    ids = torch.randint(0, V, (N,), device=DEV)
    Y, dW = Guarded((N, H), dtype), Guarded((V, H), torch.float32)
    cuda_lib.flce_embed_fwd(W, ids, out=Y.t)
    info = {}
    cuda_lib.flce_embed_bwd(W[ids], ids, V, info=info)
    ws = Guarded((info["workspace_bytes"],), torch.uint8)
    cuda_lib.flce_embed_bwd(W[ids], ids, dW=dW.t, workspace=ws.t, sync=True)
    for name, g in (("Y", Y), ("dW", dW), ("workspace", ws)):
        g.check(name)
    keep = dW.t.clone()
    cuda_lib.flce_embed_bwd(W[ids], ids, dW=dW.t, accumulate=True, workspace=ws.t, sync=True)
    for name, g in (("dW", dW), ("workspace", ws)):
        g.check(name)
    unused = torch.ones(V, dtype=torch.bool, device=DEV)
    unused[ids] = False
    assert torch.equal(dW.t[unused], keep[unused])


@pytest.mark.parametrize("lens,Hq,Hkv,D,pad", [
    ([1], 1, 1, 8, 0), ([127, 129, 0, 300], 4, 2, 64, 3), ([257], 2, 1, 128, 0),
    ([90, 400], 8, 1, 72, 1), ([128] * 5, 4, 4, 128, 0),
])
def test_attention_bounds(cuda_lib, lens, Hq, Hkv, D, pad):
    T = sum(lens) + pad
    bf = torch.bfloat16
    q, k, v = (torch.randn(T, h, D, device=DEV).to(bf) for h in (Hq, Hkv, Hkv))
    dO = torch.randn(T, Hq, D, device=DEV).to(bf)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    out = {n: Guarded((T, h, D), bf) for n, h in (("o", Hq), ("dq", Hq), ("dk", Hkv), ("dv", Hkv))}
    out["lse"] = Guarded((Hq, T), torch.float32)
    info = {}
    cuda_lib.flce_attn_fwd(q, k, v, cu, info=info)
    ws = Guarded((info["workspace_bytes"],), torch.uint8)
    cuda_lib.flce_attn_fwd(q, k, v, cu, out=out["o"].t, lse=out["lse"].t, workspace=ws.t, sync=True)
    ws.check("forward workspace")
    cuda_lib.flce_attn_bwd(dO, q, k, v, out["o"].t, out["lse"].t, cu, info=info)
    ws = Guarded((info["workspace_bytes"],), torch.uint8)
    cuda_lib.flce_attn_bwd(dO, q, k, v, out["o"].t, out["lse"].t, cu, dq=out["dq"].t,
                           dk=out["dk"].t, dv=out["dv"].t, workspace=ws.t, sync=True)
    ws.check("backward workspace")
    for name, g in out.items():
        g.check(name)


@pytest.mark.parametrize("shape", [(1, 1), (127, 129), (300, 72), (3, 130, 257), (130, 2300),
                                   (1300, 1400)])
def test_orthogonalize_bounds(cuda_lib, shape):
    G = torch.randn(*shape, device=DEV)
    out = Guarded(shape, torch.bfloat16)
    info = {}
    cuda_lib.flce_orthogonalize(G, info=info)
    ws = Guarded((info["workspace_bytes"],), torch.uint8)
    cuda_lib.flce_orthogonalize(G, out=out.t, workspace=ws.t, sync=True)
    out.check("out")
    ws.check("workspace")


def test_embed_far_rows(cuda_lib):
    """Rows beyond 2^31 elements from the table's start."""
    V, H = 530_000, 4096
    W = torch.empty(V, H, dtype=torch.bfloat16, device=DEV)
    ids = torch.tensor([V - 1, 0, 524_289, V - 1, 524_287], device=DEV)
    W[ids] = torch.randn(5, H, device=DEV).bfloat16()
    Y = cuda_lib.flce_embed_fwd(W, ids, sync=True)
    assert torch.equal(Y, W[ids])
    del W
    dW = torch.empty(V, H, device=DEV)
    old = torch.randn(5, H, device=DEV)
    dW[ids] = old
    before = dW[ids].clone()
    cuda_lib.flce_embed_bwd(Y, ids, dW=dW, accumulate=True, sync=True)
    add = Y.float()
    add[0] = add[3] = Y[0].float() + Y[3].float()
    assert torch.equal(dW[ids], before + add)


def test_attention_far_tokens(cuda_lib):
    """Token strides that put the last tokens beyond 2^31 elements."""
    T, Hq, Hkv, D, stride = 300, 2, 1, 64, 8_000_000
    raw = torch.empty(T * stride, dtype=torch.bfloat16, device=DEV)
    rows = raw.view(T, stride)
    q, k, v, dO, dq = (rows[:, a:a + h * D].view(T, h, D) for a, h in (
        (0, Hq), (1000, Hkv), (2000, Hkv), (3000, Hq), (4000, Hq)))
    for t in (q, k, v, dO):
        t.copy_(torch.randn(t.shape, device=DEV))
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device=DEV)
    o, lse = cuda_lib.flce_attn_fwd(q, k, v, cu, sync=True)
    _, dk, dv = cuda_lib.flce_attn_bwd(dO, q, k, v, o, lse, cu, dq=dq, sync=True)
    near = [t.contiguous() for t in (q, k, v, dO)]
    o2, lse2 = cuda_lib.flce_attn_fwd(*near[:3], cu)
    dq2, dk2, dv2 = cuda_lib.flce_attn_bwd(near[3], *near[:3], o2, lse2, cu)
    for a, b in ((o, o2), (lse, lse2), (dq, dq2), (dk, dk2), (dv, dv2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(2361, 2305), (2520, 4133), (4100, 2380), (2, 1300, 1405)])
def test_orthogonalize_bounds_of_pairs(cuda_lib, shape):
    """The same where the products run on CTA pairs."""
    test_orthogonalize_bounds(cuda_lib, shape)
