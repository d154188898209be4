"""Newton-Schulz orthogonalisation against the same iteration in 64 bits.

Tolerance on the relative Frobenius error: rounding the result to bf16 gives
2^-8 / sqrt(3) or less on average over mantissas, 1.7e-3 (2.3e-3 at the worst
mantissa); the fp16 operands of the products (half a step of 2^-11 each, three
roundings per step that the next steps neither damp nor amplify much, since X
itself stays in fp32) give 2e-3 in a simulation with those roundings.  5e-3
covers the sum with room for small matrices, where single entries count."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
ABC = (3.4445, -4.7750, 2.0315)
TOL = 5e-3
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _reference(G, steps=5, abc=ABC, eps=1e-7):
    a, b, c = abc
    out = []
    for g in G.double().reshape(-1, *G.shape[-2:]):
        X = g / (torch.linalg.norm(g) + eps)
        for _ in range(steps):
            if g.shape[0] <= g.shape[1]:
                A = X @ X.T
                X = a * X + (b * A + c * (A @ A)) @ X
            else:
                A = X.T @ X
                X = a * X + X @ (b * A + c * (A @ A))
        out.append(X)
    return torch.stack(out).reshape(G.shape)


def _matrix(kind, shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    *batch, m, n = shape
    noise = torch.randn(*shape, generator=g)
    if kind == "noise":
        G = noise
    else:
        r = min(8, m, n)
        low = torch.randn(*batch, m, r, generator=g) @ torch.randn(*batch, r, n, generator=g)
        G = low + noise if kind == "signal" else low  # else: of rank 8
    return (G * 1e-3).to(DT[dtype]).to(DEV)


def _check(got, ref):
    assert got.dtype == torch.bfloat16 and got.shape == ref.shape
    for x, y in zip(got.double().reshape(-1, *ref.shape[-2:]), ref.reshape(-1, *ref.shape[-2:])):
        assert (x - y).norm().item() <= TOL * y.norm().item()


@pytest.mark.parametrize("kind", ["noise", "signal", "rank8"])
@pytest.mark.parametrize("shape,dtype", [
    ((1, 1), "fp32"),
    ((1, 300), "bf16"),           # one row
    ((129, 1), "fp32"),           # one column
    ((64, 64), "bf16"),
    ((127, 129), "fp32"),         # odd rows: no whole vectors anywhere
    ((200, 72), "bf16"),          # tall
    ((333, 1001), "bf16"),
    ((1001, 333), "fp32"),
    ((3, 130, 257), "fp32"),      # stacked, odd matrix size
    ((2, 5, 40, 24), "bf16"),
    ((640, 640), "fp32"),
    ((1300, 1500), "bf16"),       # CTA pairs
    ((1500, 1290), "fp32"),
])
def test_orthogonalize(cuda_lib, shape, dtype, kind):
    G = _matrix(kind, shape, sum(shape), dtype)
    got = cuda_lib.flce_orthogonalize(G, sync=True)
    _check(got, _reference(G))
    assert torch.equal(got, cuda_lib.flce_orthogonalize(G))


@pytest.mark.parametrize("steps,abc", [(1, ABC), (2, ABC), (10, ABC), (12, (1.5, -0.5, 0.0)),
                                       (8, (1.875, -1.25, 0.375))])
def test_orthogonalize_polynomials(cuda_lib, steps, abc):
    G = _matrix("noise", (96, 400), 5, "fp32")
    got = cuda_lib.flce_orthogonalize(G, steps=steps, coeffs=abc, sync=True)
    _check(got, _reference(G, steps, abc))


def test_orthogonalize_does_not_depend_on_the_scale(cuda_lib):
    """A power of two in G changes nothing but the eps beside the norm."""
    G = _matrix("signal", (150, 260), 6, "fp32") * 1024
    ref = cuda_lib.flce_orthogonalize(G, eps=0.0)
    for s in (2.0 ** -40, 2.0 ** 30):
        assert torch.equal(cuda_lib.flce_orthogonalize(G * s, eps=0.0), ref)


def test_orthogonalize_zeros_and_nonfinite(cuda_lib):
    G = torch.zeros(3, 70, 90, device=DEV)
    G[1] = torch.randn(70, 90, device=DEV)
    G[2] = torch.randn(70, 90, device=DEV)
    G[2, 3, 4] = float("nan")
    got = cuda_lib.flce_orthogonalize(G, sync=True)
    assert not got[0].any()                       # zeros stay zeros
    _check(got[1:2], _reference(G[1:2]))          # a NaN next door changes nothing
    assert bool(got[2].isnan().all())             # and spreads over its own matrix


def test_orthogonalize_empty(cuda_lib):
    for shape in ((0, 5), (5, 0), (0, 4, 4)):
        assert cuda_lib.flce_orthogonalize(torch.empty(shape, device=DEV), sync=True).shape == shape


def test_orthogonalize_side_stream_and_workspace(cuda_lib):
    G = _matrix("noise", (2, 140, 300), 7, "bf16")
    info = {}
    ref = cuda_lib.flce_orthogonalize(G, info=info)
    assert int(info["status"].item()) == 0
    ws = torch.empty(info["workspace_bytes"], dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cuda_lib.flce_orthogonalize(G, workspace=ws)
    side.synchronize()
    assert torch.equal(got, ref)
    with pytest.raises(cuda_lib.FlceError) as e:
        cuda_lib.flce_orthogonalize(G, workspace=ws[:-256])
    assert e.value.status == cuda_lib.FLCE_ERR_WORKSPACE


def test_orthogonalize_in_a_graph(cuda_lib):
    G = _matrix("noise", (200, 500), 8, "fp32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # per-device setup outside the capture
        cuda_lib.flce_orthogonalize(G)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cuda_lib.flce_orthogonalize(G)
    for seed in (9, 10):
        G.copy_(_matrix("signal", (200, 500), seed, "fp32"))
        graph.replay()
        assert torch.equal(out, cuda_lib.flce_orthogonalize(G))


def test_orthogonalize_refusals(cuda_lib):
    G = torch.randn(8, 16, device=DEV)
    for bad in (G.half(), G[0], G.T, G.cpu()):
        with pytest.raises((ValueError, TypeError)):
            cuda_lib.flce_orthogonalize(bad)
    with pytest.raises(ValueError):
        cuda_lib.flce_orthogonalize(G, out=torch.empty(8, 16, device=DEV))
    with pytest.raises(cuda_lib.FlceError):
        cuda_lib.flce_orthogonalize(G, coeffs=(5.0, 0.0, 0.0))


@pytest.mark.parametrize("shape,dtype", [
    ((260, 2300), "fp32"),        # X X^T with its long K shared out over four CTAs
    ((2500, 129), "bf16"),
    ((2, 100, 2049), "fp32"),
    ((900, 2100), "bf16"),        # as many tiles as that shape takes
])
def test_orthogonalize_long_products(cuda_lib, shape, dtype):
    G = _matrix("signal", shape, sum(shape), dtype)
    got = cuda_lib.flce_orthogonalize(G, sync=True)
    _check(got, _reference(G))
    assert torch.equal(got, cuda_lib.flce_orthogonalize(G))


@pytest.mark.parametrize("shape,dtype", [
    ((256, 256), "fp32"),
    ((255, 1000), "bf16"),
    ((192, 193), "fp32"),         # three K blocks, a second half of 64 rows
    ((700, 65), "bf16"),          # tall
    ((1, 5000), "fp32"),
    ((300, 40, 24), "bf16"),      # two rounds of CTAs
    ((9000, 250), "fp32"),
    ((5, 256, 7001), "bf16"),     # more: products of their own
    ((257, 300), "fp32"),         # just past it
])
def test_orthogonalize_small_side(cuda_lib, shape, dtype):
    """The second and third product in one launch."""
    G = _matrix("signal", shape, sum(shape) + 1, dtype)
    got = cuda_lib.flce_orthogonalize(G, sync=True)
    _check(got, _reference(G))
    assert torch.equal(got, cuda_lib.flce_orthogonalize(G))


@pytest.mark.parametrize("shape", [(150, 260), (2, 90, 33), (700, 640)])
@pytest.mark.parametrize("power", [-126, -110, -75, 50, 64, 100, 123])
def test_orthogonalize_far_scales(cuda_lib, shape, power):
    """Powers of two whose squares fp32 does not hold: the same bits."""
    G = _matrix("noise", shape, 11, "fp32") * 1024
    G = torch.where(G.abs() < 2.0 ** -14, G.sign() * 2.0 ** -14, G)  # no entry becomes subnormal
    s = 2.0 ** power if power > -112 else 2.0 ** (power + 14)
    ref = cuda_lib.flce_orthogonalize(G, eps=0.0)
    assert torch.equal(cuda_lib.flce_orthogonalize(G * s, eps=0.0, sync=True), ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_orthogonalize_extreme_entries(cuda_lib, dtype):
    """The largest entries, subnormal ones, and both in one matrix."""
    G = _matrix("noise", (120, 333), 12, "fp32") * 1000
    top = torch.finfo(DT[dtype]).max
    big = (G / G.abs().max() * top).to(DT[dtype])
    assert bool(big.isfinite().all())
    small = (G * 2.0 ** -132).to(DT[dtype])
    spread = G.to(DT[dtype])
    spread[5, 7], spread[50, 300] = top, -top / 2
    both = torch.stack([big, small, spread])
    got = cuda_lib.flce_orthogonalize(both, eps=0.0, sync=True)
    _check(got, _reference(both, eps=0.0))
    # the eps counts beside a norm of its own size only
    _check(cuda_lib.flce_orthogonalize(big, eps=1.0), _reference(big, eps=1.0))


def shapes_of(lib, shape, sms):
    """The tile shapes of a step's three products."""
    batch = 1
    for n in shape[:-2]:
        batch *= n
    out = (ctypes.c_int32 * 3)()
    assert lib.flce_selftest_ortho_shapes(batch, *shape[-2:], sms, out) == 0
    return tuple(out)


PAIR, SINGLE, SPLIT, MERGED = range(4)
FORMS = [
    # last tile of 256 with one row; update tiles in one round of single CTAs
    ((2361, 2305), "fp32", (PAIR, PAIR, SINGLE)),
    # tall, every product on pairs, more than two tiles per pair; 76 rows in the last tile
    ((4100, 2380), "bf16", (PAIR, PAIR, PAIR)),
    # 216 rows there: some of the odd CTA's; no whole vectors
    ((2520, 4133), "fp32", (PAIR, PAIR, PAIR)),
    ((3, 1300, 1500), "bf16", (PAIR, PAIR, SINGLE)),
    ((900, 2100), "fp32", (SPLIT, SINGLE, SINGLE)),
    ((640, 640), "bf16", (SINGLE, SINGLE, SINGLE)),
    ((8, 250, 1030), "bf16", (SINGLE, MERGED, MERGED)),
]


@pytest.mark.parametrize("shape,dtype,forms", FORMS)
def test_orthogonalize_forms(cuda_lib, shape, dtype, forms):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert shapes_of(cuda_lib.load_library(), shape, sms) == forms
    G = _matrix("signal", shape, sum(shape) + 2, dtype)
    got = cuda_lib.flce_orthogonalize(G, sync=True)
    _check(got, _reference(G))
    assert torch.equal(got, cuda_lib.flce_orthogonalize(G))
