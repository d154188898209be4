"""8-bit checkpoints bit for bit against the definition, and the weight gradient from them.

Tolerance of the weight gradient.  Products of a bf16 dY and a stored x are exact in fp32.
A sum over N tokens adds at most N of them and each addition, rounded or cut off, is off by
at most 2^-23 of a partial sum, which is at most A = sum |dY x|; the old value is added last:
(N + 16) 2^-23 A + 2^-23 |old| bounds the error.  Its 2-norm over the matrix is far
smaller: terms of random sign make partial sums of about sqrt(k / N) of the result, so that
even additions that always cut off (half a unit on average, one for every 16 tokens) take
about N / 16 * 2^-24 * 2 / 3 of it; 1e-5 is what the sums are held to here, whatever N."""
import pytest
import torch

import block_util as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def _x(N, H, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * N + H)
    x = torch.randn(N, H, generator=g) * torch.exp(3 * torch.randn(N, 1, generator=g))
    x[torch.rand(N, H, generator=g) < 0.05] = 0
    return x.to(dtype)


def _bytes(x):
    codes, scales = ref.quantise(x)
    return torch.cat([codes.view(-1), scales.view(-1)])


@pytest.mark.parametrize("N,H", [(1, 8), (3, 32), (5, 40), (33, 136), (7, 1000), (130, 4096),
                                 (2, 20000), (1001, 64)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_save_and_load(cuda_lib, N, H, dtype):
    x = _x(N, H, dtype)
    ck = cuda_lib.Checkpoint.empty(N, H, DEV)
    ck.data.fill_(0xA5)
    cuda_lib.flce_ckpt_save(x.to(DEV), out=ck, sync=True)
    want = _bytes(x)
    assert torch.equal(ck.data.cpu(), want)
    back = ref.dequantise(*ref.quantise(x), H)
    for dt in (BF, FP):
        got = cuda_lib.flce_ckpt_load(ck, dtype=dt, sync=True)
        assert torch.equal(got.cpu().double(), back)  # exact in bf16 too


def test_every_value(cuda_lib):
    """All bf16 numbers, as the largest of their group and beside larger ones; ties, subnormals,
    infinities and NaN; signed zeros."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    alone = torch.zeros(65536, 32, dtype=BF)
    alone[:, 5] = every
    beside = every.view(2048, 32)
    g = torch.Generator().manual_seed(0)
    mixed = every[torch.randperm(65536, generator=g)].view(2048, 32)
    ties = (torch.arange(4096).float() * 0.0625 - 100).to(BF).view(-1, 64)
    for x in (alone, beside, mixed, ties, beside.flip(1).reshape(1024, 64)):
        codes, scales = ref.quantise(x)
        ck = cuda_lib.flce_ckpt_save(x.to(DEV), sync=True)
        got = ck.data.cpu()
        assert torch.equal(got[codes.numel():], scales.view(-1))
        nan = (scales[:, :codes.shape[1] // 32] == 255).repeat_interleave(32, 1)
        assert torch.equal(got[:codes.numel()].view(codes.shape)[~nan], codes[~nan])
        back = ref.dequantise(codes, scales, x.shape[1])
        for dt in (BF, FP):
            assert torch.equal(cuda_lib.flce_ckpt_load(ck, dtype=dt).cpu().double().nan_to_num(7.0),
                               back.nan_to_num(7.0))


def test_fp32_range(cuda_lib):
    """fp32 subnormals, numbers beyond bf16's largest, and ties of the scale."""
    x = torch.zeros(6, 64)
    x[0, :4] = torch.tensor([1e-45, 1e-40, -1e-38, 3e-38])
    x[1, :4] = torch.tensor([3.4028234e38, -3.39e38, 1e38, 1.0])
    x[2, :3] = torch.tensor([448.0, 448.00003, 1.0])
    x[3, :3] = torch.tensor([448.0, 447.99997, 17.0])
    x[4, :2] = torch.tensor([float("inf"), 1.0])
    x[5, 33] = float("nan")
    ck = cuda_lib.flce_ckpt_save(x.to(DEV), sync=True)
    codes, scales = ref.quantise(x)
    keep = (scales[:, :2] != 255).repeat_interleave(32, 1)
    got = ck.data.cpu()
    assert torch.equal(got[codes.numel():], scales.view(-1))
    assert torch.equal(got[:codes.numel()].view(codes.shape)[keep], codes[keep])
    back = cuda_lib.flce_ckpt_load(ck, dtype=FP).cpu()
    assert bool(back[4, :32].isnan().all()) and not back[4, 32:].any()
    assert bool(back[5, 32:].isnan().all()) and not back[5, :32].any()
    assert back[1, 0] == 1.75 * 2.0 ** 127


def test_strides(cuda_lib):
    x = _x(50, 200, BF).to(DEV)
    wide = torch.full((50, 264), 3.0, dtype=BF, device=DEV)
    wide[:, 8:208] = x
    ck = cuda_lib.flce_ckpt_save(wide[:, 8:208])
    assert torch.equal(ck.data, cuda_lib.flce_ckpt_save(x).data)
    cuda_lib.flce_ckpt_load(ck, out=wide[:, 16:216])
    assert torch.equal(wide[:, 16:216], cuda_lib.flce_ckpt_load(ck))
    assert bool((wide[:, 216:] == 3).all())


def test_fp32_rows_at_any_16_bytes(cuda_lib):
    """Rows that begin on a multiple of 32 bytes, and those that do not."""
    ck = cuda_lib.flce_ckpt_save(_x(70, 136, FP).to(DEV))
    want = cuda_lib.flce_ckpt_load(ck, dtype=FP)
    for at in (0, 4, 8, 12):
        buf = torch.full((70, 160), 3.0, device=DEV)
        cuda_lib.flce_ckpt_load(ck, out=buf[:, at:at + 136])
        assert torch.equal(buf[:, at:at + 136], want)
        assert bool((buf[:, :at] == 3).all()) and bool((buf[:, at + 136:] == 3).all())


def _check_wgrad(got, dY, x, old):
    dY, x = dY.double(), x.double()
    want, A = dY.t() @ x, dY.t().abs() @ x.abs()
    if old is not None:
        want, A = want + old.double(), A + old.double().abs()
    err = got.double() - want
    assert bool((err.abs() <= (dY.shape[0] + 17) * 2.0 ** -23 * A).all())
    assert err.norm() <= 1e-5 * want.norm()


@pytest.mark.parametrize("N,O,I", [
    (1, 8, 8), (5, 64, 40), (64, 256, 256), (65, 264, 136), (130, 520, 392), (1000, 8, 1000),
    (333, 1000, 24), (2049, 512, 520), (4100, 264, 264)])
def test_wgrad(cuda_lib, N, O, I):
    g = torch.Generator().manual_seed(N)
    dY = torch.randn(N, O, generator=g).to(BF).to(DEV)
    ck = cuda_lib.flce_ckpt_save(_x(N, I, BF).to(DEV))
    x = cuda_lib.flce_ckpt_load(ck)
    dW = torch.full((O, I), float("nan"), device=DEV)
    cuda_lib.flce_ckpt_wgrad(dY, ck, dW=dW, sync=True)
    _check_wgrad(dW, dY, x, None)
    assert torch.equal(cuda_lib.flce_ckpt_wgrad(dY, ck), dW)
    old = torch.randn(O, I, generator=g).to(DEV)
    acc = old.clone()
    info = {}
    cuda_lib.flce_ckpt_wgrad(dY, ck, dW=acc, accumulate=True, info=info)
    _check_wgrad(acc, dY, x, old)
    assert int(info["status"].item()) == 0
    # rows of dY in a wider buffer whose other columns are NaN
    wide = torch.full((N, O + 16), float("nan"), dtype=BF, device=DEV)
    wide[:, 8:8 + O] = dY
    assert torch.equal(cuda_lib.flce_ckpt_wgrad(wide[:, 8:8 + O], ck), dW)


@pytest.mark.parametrize("N,O,I", [
    (20001, 264, 264),    # 6 tiles of 128 columns, each shared by many CTA pairs
    (8200, 520, 2056),    # 51 tiles of 128, not shared
    (9000, 2568, 2056),   # 99 tiles of 256: a whole round and 23 that are shared
    (30000, 8, 8),        # one tile
    (2500, 3400, 3000),   # 168 tiles of 256, two whole rounds and 16 that are not shared out
    (8192, 2600, 1000),   # 44 tiles of 256, all shared
    (3040, 2976, 1624),   # 156 tiles of 128, of which 4 are shared
    (14, 5656, 2056)])    # 391 tiles of 128, five rounds
def test_wgrad_shared_tiles(cuda_lib, N, O, I):
    """Either width of tiles, and tiles that several CTA pairs share along the tokens."""
    g = torch.Generator(device=DEV).manual_seed(N)
    dY = torch.randn(N, O, generator=g, device=DEV).to(BF)
    x = torch.randn(N, I, generator=g, device=DEV).to(BF)
    ck = cuda_lib.flce_ckpt_save(x)
    x = cuda_lib.flce_ckpt_load(ck)
    dW = torch.full((O, I), float("nan"), device=DEV)
    cuda_lib.flce_ckpt_wgrad(dY, ck, dW=dW, sync=True)
    _check_wgrad(dW, dY, x, None)
    assert torch.equal(cuda_lib.flce_ckpt_wgrad(dY, ck), dW)
    old = torch.randn(O, I, generator=g, device=DEV)
    acc = old.clone()
    info = {}
    cuda_lib.flce_ckpt_wgrad(dY, ck, dW=acc, accumulate=True, info=info)
    _check_wgrad(acc, dY, x, old)
    assert int(info["status"].item()) == 0
    ws = torch.full((info["workspace_bytes"],), 0xFF, dtype=torch.uint8, device=DEV)  # NaN
    assert torch.equal(cuda_lib.flce_ckpt_wgrad(dY, ck, workspace=ws), dW)


def test_wgrad_every_scale(cuda_lib):
    """Scales over their whole range in one row: each column's products are exact, and one
    token's gradient is its product."""
    H = 32 * 237
    x = torch.zeros(1, H)
    codes = ref.e4m3_table()[:127].float()
    for i in range(237):
        e = i - 117
        x[0, 32 * i] = 448.0 * 2.0 ** e
        x[0, 32 * i + 1:32 * i + 32] = -codes[(31 * i + torch.arange(31)) % 127] * 2.0 ** e
    ck = cuda_lib.flce_ckpt_save(x.to(DEV), sync=True)
    assert torch.equal(cuda_lib.flce_ckpt_load(ck, dtype=FP).cpu(), x)
    dY = torch.tensor([[1.0, -0.5, 0, 0, 0, 0, 0, 2.0 ** -8]], dtype=BF, device=DEV)
    dW = cuda_lib.flce_ckpt_wgrad(dY, ck, sync=True).cpu()
    normal = x[0].abs() >= 2.0 ** -117  # times 2^-8 still a normal number
    assert torch.equal(dW[0], x[0]) and torch.equal(dW[1][normal], -0.5 * x[0][normal])
    assert torch.equal(dW[7][normal], x[0][normal] * 2.0 ** -8) and not dW[2:7].any()


def test_wgrad_nan(cuda_lib):
    """A NaN of the input reaches its group's columns, one of dY its row, and no others."""
    N, O, I = 300, 264, 328
    g = torch.Generator().manual_seed(1)
    dY, x = torch.randn(N, O, generator=g).to(BF), torch.randn(N, I, generator=g).to(BF)
    x[299, 70], x[3, 327], dY[7, 263] = float("nan"), float("inf"), float("nan")
    dW = cuda_lib.flce_ckpt_wgrad(dY.to(DEV), cuda_lib.flce_ckpt_save(x.to(DEV))).cpu()
    bad = torch.zeros(O, I, dtype=torch.bool)
    bad[:, 64:96] = bad[:, 320:] = bad[263] = True
    assert torch.equal(dW.isnan(), bad)


def test_wgrad_empty(cuda_lib):
    dY = torch.empty(0, 64, dtype=BF, device=DEV)
    ck = cuda_lib.flce_ckpt_save(torch.empty(0, 40, dtype=BF, device=DEV), sync=True)
    assert cuda_lib.flce_ckpt_load(ck, sync=True).shape == (0, 40)
    old = torch.randn(64, 40, device=DEV)
    keep = old.clone()
    cuda_lib.flce_ckpt_wgrad(dY, ck, dW=old, accumulate=True, sync=True)
    assert torch.equal(old, keep)
    cuda_lib.flce_ckpt_wgrad(dY, ck, dW=old, sync=True)
    assert not old.any()


def test_binding_refusals(cuda_lib):
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    ck = cuda_lib.flce_ckpt_save(x)
    for err, call in [
            (TypeError, lambda: cuda_lib.flce_ckpt_save(x.half())),
            (ValueError, lambda: cuda_lib.flce_ckpt_save(x.t())),
            (ValueError, lambda: cuda_lib.flce_ckpt_save(x, out=cuda_lib.Checkpoint.empty(4, 32, DEV))),
            (TypeError, lambda: cuda_lib.flce_ckpt_load(ck, dtype=torch.float16)),
            (ValueError, lambda: cuda_lib.flce_ckpt_load(ck, out=x[:3])),
            (ValueError, lambda: cuda_lib.Checkpoint(ck.data[:-1], 4, 64)),
            (TypeError, lambda: cuda_lib.flce_ckpt_wgrad(x.float(), ck)),
            (ValueError, lambda: cuda_lib.flce_ckpt_wgrad(x[:3], ck)),
            (ValueError, lambda: cuda_lib.flce_ckpt_wgrad(x, ck, accumulate=True)),
            (ValueError, lambda: cuda_lib.flce_ckpt_wgrad(x, ck, dW=torch.zeros(64, 63, device=DEV))),
            (TypeError, lambda: cuda_lib.CheckpointedLinear()(x.float(), x))]:
        with pytest.raises(err):
            call()


def test_linear_refuses_what_its_backward_pass_could_not_take(cuda_lib):
    """In the forward pass, not when the gradients are due."""
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    linear = cuda_lib.CheckpointedLinear()
    for w in (torch.zeros(12, 64, dtype=BF, device=DEV), torch.zeros(64, dtype=BF, device=DEV),
              torch.zeros(16, 72, dtype=BF, device=DEV)):
        with pytest.raises(ValueError):
            linear(x, w)
    with pytest.raises(ValueError):
        linear(x[:, :20], torch.zeros(16, 20, dtype=BF, device=DEV))
    with pytest.raises(ValueError):
        linear(x[0, 0], torch.zeros(16, 64, dtype=BF, device=DEV))
    w = torch.zeros(16, 64, dtype=BF, device=DEV, requires_grad=True)
    out = linear(x[:0], w)
    out.sum().backward()
    assert out.shape == (0, 16) and not w.grad.any()
