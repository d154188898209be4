"""Embedding lookup and its gradient against 64-bit sums.

Tolerances.  The lookup rounds scale * w to fp32 and then once to the output
type, which torch's fp32 product and cast do too: equal bits.  A gradient row
is a sum of n fp32 terms (each addition off by at most 2^-24 of a partial sum,
and partial sums are at most A = sum |dY|), times the scale, plus the old
value: off by at most (n + 2) 2^-24 (|scale| A + |old|)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
IGN = -100
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _ids(kind, N, V, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        ids = torch.randint(0, V, (N,), generator=g)
    elif kind == "skewed":  # frequencies like 1/rank: runs of hundreds of equal ids
        ids = (torch.exp(torch.rand(N, generator=g, dtype=torch.float64)
                         * torch.log(torch.tensor(float(V)))).long() - 1).clamp(0, V - 1)
        ids = ids * 7919 % V
    elif kind == "one":     # every token the same row
        ids = torch.full((N,), V - 1)
    elif kind == "two":     # the first and the last row, in turn
        ids = torch.arange(N) % 2 * (V - 1)
    else:                   # nothing takes part
        return torch.full((N,), IGN).to(dtype)
    ids[torch.rand(N, generator=g) < 0.1] = IGN
    return ids.to(dtype)


def _check_bwd(got, dY, ids, V, scale, old):
    dY, ids = dY.cpu().double(), ids.cpu().long()
    keep = ids != IGN
    ref = torch.zeros(V, dY.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(ref)
    ref.index_add_(0, ids[keep], dY[keep])
    mag.index_add_(0, ids[keep], dY[keep].abs())
    n = torch.bincount(ids[keep], minlength=V)[:, None].double()
    ref, mag = ref * scale, mag * abs(scale)
    if old is not None:
        ref, mag = ref + old.cpu().double(), mag + old.cpu().double().abs()
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= (n + 2) * 2.0 ** -24 * mag).all()), err.max().item()


@pytest.mark.parametrize("N,H,V,dtype,scale,idt", [
    (1, 8, 1, "bf16", 1.0, torch.int64),
    (7, 4, 5, "fp32", 3.0, torch.int32),
    (300, 1000, 777, "bf16", 0.3, torch.int64),
    (1025, 4096, 5003, "bf16", 64.0, torch.int32),
    (333, 1028, 50, "fp32", -1.7, torch.int64),
])
def test_embed_fwd(cuda_lib, N, H, V, dtype, scale, idt):
    W = torch.randn(V, H, generator=torch.Generator().manual_seed(N)).to(DT[dtype]).to(DEV)
    ids = _ids("uniform", N, V, N + 1, idt).to(DEV)
    info = {}
    Y = cuda_lib.flce_embed_fwd(W, ids, scale=scale, info=info)
    s = torch.tensor(scale, dtype=torch.float32, device=DEV)
    ref = (W[ids.long().clamp(min=0)].float() * s).masked_fill((ids == IGN)[:, None], 0).to(W.dtype)
    assert torch.equal(Y, ref)
    assert int(info["status"].item()) == 0


@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "two", "none"])
@pytest.mark.parametrize("N,H,V,dtype,scale", [
    (1, 8, 3, "bf16", 1.0),
    (5, 4, 2, "fp32", 0.5),
    (257, 1000, 600, "bf16", 1.0),       # one radix pass less than two full digits
    (3001, 136, 32003, "fp32", 45.25),   # two passes
    (4100, 4104, 300, "bf16", -0.25),    # more than one slice of a row
    (20000, 64, 300000, "bf16", 1.0),    # three passes of digits, chunks of many tokens
])
def test_embed_bwd(cuda_lib, N, H, V, dtype, scale, kind):
    g = torch.Generator().manual_seed(N + H)
    dY = torch.randn(N, H, generator=g).to(DT[dtype]).to(DEV)
    ids = _ids(kind, N, V, N + 2, torch.int32 if N % 2 else torch.int64).to(DEV)
    dense = torch.full((V, H), float("nan"), device=DEV)
    cuda_lib.flce_embed_bwd(dY, ids, V, scale=scale, dW=dense, sync=True)
    _check_bwd(dense, dY, ids, V, scale, None)
    old = torch.randn(V, H, generator=g).to(DEV)
    acc = old.clone()
    cuda_lib.flce_embed_bwd(dY, ids, scale=scale, dW=acc, accumulate=True)
    _check_bwd(acc, dY, ids, V, scale, old)
    used = torch.zeros(V, dtype=torch.bool, device=DEV)
    used[ids[ids != IGN].long()] = True
    assert torch.equal(acc[~used], old[~used])
    again = cuda_lib.flce_embed_bwd(dY, ids, V, scale=scale)
    assert torch.equal(again, dense)  # the order of the sums does not change


def test_embed_empty(cuda_lib):
    W = torch.randn(5, 8, device=DEV)
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    assert cuda_lib.flce_embed_fwd(W, ids, sync=True).shape == (0, 8)
    dY = torch.empty(0, 8, device=DEV)
    assert torch.equal(cuda_lib.flce_embed_bwd(dY, ids, 5, sync=True), torch.zeros(5, 8, device=DEV))
    old = torch.randn(5, 8, device=DEV)
    keep = old.clone()
    cuda_lib.flce_embed_bwd(dY, ids, dW=old, accumulate=True, sync=True)
    assert torch.equal(old, keep)


def test_embed_bad_ids(cuda_lib):
    """Ids outside the table read and write nothing: zero rows, no gradient, an error."""
    W = torch.randn(50, 64, device=DEV)
    ids = torch.tensor([3, 50, -1, 2 ** 31 + 3, 7, -(2 ** 40), IGN], device=DEV)
    bad = torch.tensor([False, True, True, True, False, True, True], device=DEV)
    info = {}
    Y = cuda_lib.flce_embed_fwd(W, ids, info=info)
    assert int(info["status"].item()) == cuda_lib.FLCE_ERR_TARGET
    assert torch.equal(Y[~bad], W[ids[~bad]]) and not Y[bad].any()
    with pytest.raises(cuda_lib.FlceError) as e:
        cuda_lib.flce_embed_fwd(W, ids, sync=True)
    assert e.value.status == cuda_lib.FLCE_ERR_TARGET
    dY = torch.randn(7, 64, device=DEV)
    dW = cuda_lib.flce_embed_bwd(dY, ids, 50, info=info)
    assert int(info["status"].item()) == cuda_lib.FLCE_ERR_TARGET
    ref = torch.zeros(50, 64, device=DEV)
    ref[3], ref[7] = dY[0], dY[4]
    assert torch.equal(dW, ref)


def test_embed_nonfinite_rows_stay_theirs(cuda_lib):
    """An infinite or NaN gradient row reaches its own row of dW only."""
    dY = torch.ones(6, 16, device=DEV)
    dY[1], dY[4] = float("inf"), float("nan")
    ids = torch.tensor([0, 1, 2, 0, IGN, 2], device=DEV)
    dW = cuda_lib.flce_embed_bwd(dY, ids, 4)
    ref = torch.tensor([2.0, float("inf"), 2.0, 0.0], device=DEV)[:, None].expand(4, 16)
    assert torch.equal(dW, ref)


def test_embed_side_stream_and_workspace(cuda_lib):
    N, H, V = 2000, 256, 900
    dY = torch.randn(N, H, device=DEV)
    ids = _ids("skewed", N, V, 4).to(DEV)
    info = {}
    ref = cuda_lib.flce_embed_bwd(dY, ids, V, info=info)
    ws = torch.empty(info["workspace_bytes"], dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cuda_lib.flce_embed_bwd(dY, ids, V, workspace=ws)
    side.synchronize()
    assert torch.equal(got, ref)
    with pytest.raises(cuda_lib.FlceError) as e:
        cuda_lib.flce_embed_bwd(dY, ids, V, workspace=ws[:-256])
    assert e.value.status == cuda_lib.FLCE_ERR_WORKSPACE


def test_embed_in_a_graph(cuda_lib):
    N, H, V = 700, 128, 400
    W = torch.randn(V, H, device=DEV).bfloat16()
    ids = _ids("skewed", N, V, 5).to(DEV)
    dW = torch.zeros(V, H, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # per-device setup outside the capture
        cuda_lib.flce_embed_bwd(cuda_lib.flce_embed_fwd(W, ids), ids, dW=dW)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = cuda_lib.flce_embed_fwd(W, ids, scale=2.0)
        cuda_lib.flce_embed_bwd(Y, ids, dW=dW)
    for seed in (6, 7):
        ids.copy_(_ids("skewed", N, V, seed).to(DEV))
        graph.replay()
        Ye = cuda_lib.flce_embed_fwd(W, ids, scale=2.0)
        assert torch.equal(Y, Ye)
        assert torch.equal(dW, cuda_lib.flce_embed_bwd(Ye, ids, V))


def test_embed_module_gradient(cuda_lib):
    """Autograd: the gradient is the formula's, and that of the linear map by differences."""
    V, H, N = 40, 32, 90
    W = torch.randn(V, H, device=DEV, requires_grad=True)
    ids = _ids("uniform", N, V, 8).to(DEV)
    C = torch.randn(N, H, device=DEV)
    emb = cuda_lib.Embedding(scale=1.5)
    f = (emb(W, ids) * C).sum()
    f.backward()
    _check_bwd(W.grad, C, ids, V, 1.5, None)
    D = torch.randn(V, H, device=DEV)
    with torch.no_grad():
        plus = (emb(W + D, ids).double() * C.double()).sum()
        minus = (emb(W - D, ids).double() * C.double()).sum()
    # linear in W: the difference is exact up to the roundings of N * H products
    slope = (W.grad.double() * D.double()).sum()
    size = ((emb(W + D, ids).double() * C.double()).abs().sum()
            + (emb(W - D, ids).double() * C.double()).abs().sum())
    assert abs(((plus - minus) / 2 - slope).item()) <= 4 * N * 2.0 ** -24 * size.item()


def test_tied_weight_accumulates_on_the_head(cuda_lib):
    """dW of the head and the embedding's gradient in one fp32 buffer."""
    from flce_synth import make_case
    X, W, t = make_case(300, 64, 500, "bf16", seed=9, ignore_num=10)
    X, W, t = X.to(DEV), W.to(DEV), t.to(DEV)
    _, _, dX, dW = cuda_lib.flce_fwd_bwd_ex(X, W, t, IGN, sync=True)
    head = dW.clone()
    cuda_lib.flce_embed_bwd(dX, t, dW=dW, accumulate=True)
    _check_bwd(dW, dX, t, 500, 1.0, head)


@pytest.mark.parametrize("N,H,V,dtype,kind", [
    (1, 1024, 50003, "bf16", "two"),
    (9, 1024, 50003, "bf16", "none"),
    (700, 1000, 50521, "fp32", "skewed"),
    (3001, 1024, 50003, "bf16", "uniform"),
    (9001, 1024, 50003, "bf16", "skewed"),
    (2500, 8, 6300001, "bf16", "uniform"),      # many rows per clearing CTA
    (33, 65544, 801, "fp32", "uniform"),        # less than one
])
def test_embed_bwd_large_tables(cuda_lib, N, H, V, dtype, kind):
    """dW of more than 192 MiB, cleared in two parts: it holds NaN before, and each
    row without a token is exactly zero after."""
    ids = _ids(kind, N, V, N).to(DEV)
    dY = torch.randn(N, H, generator=torch.Generator().manual_seed(N + 1)).to(DT[dtype]).to(DEV)
    dW = torch.full((V, H), float("nan"), device=DEV)
    assert dW.numel() * 4 > 192 << 20
    cuda_lib.flce_embed_bwd(dY, ids, V, dW=dW, scale=0.5)
    keep = ids != IGN
    rows, where, n = torch.unique(ids[keep], return_inverse=True, return_counts=True)
    ref = torch.zeros(rows.numel(), H, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    ref.index_add_(0, where, dY[keep].double())
    mag.index_add_(0, where, dY[keep].double().abs())
    err = (dW[rows].double() - 0.5 * ref).abs()
    assert bool((err <= (n[:, None] + 2) * 2.0 ** -24 * 0.5 * mag).all())
    dW[rows] = 0.0
    assert bool((dW == 0).all())


def _check_rows(dW, dY, ids, scale):
    """As _check_bwd, on the GPU and for the rows that have tokens; the others are zero."""
    keep = ids != IGN
    rows, where, n = torch.unique(ids[keep], return_inverse=True, return_counts=True)
    ref = torch.zeros(rows.numel(), dY.shape[1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    ref.index_add_(0, where, dY[keep].double())
    mag.index_add_(0, where, dY[keep].double().abs())
    err = (dW[rows].double() - scale * ref).abs()
    assert bool((err <= (n[:, None] + 2) * 2.0 ** -24 * abs(scale) * mag).all())
    assert int(dW.any(1).sum()) <= rows.numel() and not dW.isnan().any()


@pytest.mark.parametrize("kind", ["uniform", "skewed", "one"])
@pytest.mark.parametrize("N", [2048, 2049, 4096, 4097])
def test_embed_bwd_sort_limits(cuda_lib, N, kind):
    """Around the token counts that one CTA sorts, with a dW that makes it the choice up
    to 4096 tokens (64 to 192 MiB to clear), and the scratch of either form."""
    H, V = 1024, 17000
    assert 64 << 20 <= V * H * 4 < 192 << 20
    ids = _ids(kind, N, V, N).to(DEV)
    dY = torch.randn(N, H, generator=torch.Generator().manual_seed(N)).bfloat16().to(DEV)
    dense, tied = {}, {}
    dW = torch.full((V, H), float("nan"), device=DEV)
    cuda_lib.flce_embed_bwd(dY, ids, V, dW=dW, scale=0.5, info=dense)
    assert int(dense["status"].item()) == 0
    _check_rows(dW, dY, ids, 0.5)
    acc = torch.zeros(V, H, device=DEV)
    cuda_lib.flce_embed_bwd(dY, ids, dW=acc, accumulate=True, scale=0.5, info=tied)
    assert torch.equal(acc, dW)  # the other sort, the same order
    lists = 2 * -(-8 * N // 256) * 256
    assert tied["workspace_bytes"] - dense["workspace_bytes"] == (lists if 2048 < N <= 4096 else 0)
    ws = torch.empty(dense["workspace_bytes"], dtype=torch.uint8, device=DEV)
    again = cuda_lib.flce_embed_bwd(dY, ids, V, scale=0.5, workspace=ws)
    assert torch.equal(again, dW)


@pytest.mark.parametrize("kind", ["uniform", "skewed", "one"])
@pytest.mark.parametrize("N,H,V,dtype", [(65536, 256, 5003, "bf16"), (130001, 72, 128256, "fp32")])
def test_embed_bwd_many_tokens(cuda_lib, N, H, V, dtype, kind):
    """The long-context batch: runs of up to N equal ids, many passes of each CTA's sort."""
    ids = _ids(kind, N, V, N, torch.int32 if N % 2 else torch.int64).to(DEV)
    dY = torch.randn(N, H, generator=torch.Generator().manual_seed(N)).to(DT[dtype]).to(DEV)
    dW = torch.full((V, H), float("nan"), device=DEV)
    cuda_lib.flce_embed_bwd(dY, ids, V, dW=dW, scale=2.0, sync=True)
    _check_rows(dW, dY, ids.long(), 2.0)
    acc = torch.zeros(V, H, device=DEV)
    cuda_lib.flce_embed_bwd(dY, ids, dW=acc, accumulate=True, scale=2.0)
    assert torch.equal(acc, dW)
