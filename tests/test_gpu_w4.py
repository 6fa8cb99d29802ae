"""GPU parity of the 4-bit weights' quantiser and matrix-vector product (twell_w4_quantize, twell_w4_matvec).

The quantiser's codes and scales equal the definition's (fp32) exactly. The product: x and code - 8 enter
exactly, every product is exact in fp32, a group's sum and the sum over groups are fp32; a sum of k terms in any
order and with truncating additions stays within k 2^-22 sum|x w|, and y is rounded once to bf16 (2^-8)."""
import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()
    binding.status_buffer(cuda_dev).zero_()
    yield
    assert binding.twell_read_status() == 0, "device status was raised"


def _weights(dev, n, k, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    W = torch.randn((n, k), generator=g) * torch.exp(torch.randn((n, 1), generator=g)) / k ** 0.5
    return W.to(BF).to(dev)


def _define(W, group):
    n, k = W.shape
    w = W.float().view(n, k // group, group)
    a = w.abs().amax(-1)
    s = (a / torch.full_like(a, 7.0)).to(BF)
    q = torch.where(s[..., None] > 0, torch.round(w / s.float()[..., None]).clamp(-8, 7), torch.zeros_like(w))
    return q, s


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 128), (8, 256), (16, 384), (33, 640), (130, 2048), (5, 896)])
def test_quantize(cuda_dev, n, k, group):
    W = _weights(cuda_dev, n, k, n + k)
    W[0, :group] = 0
    P = binding.twell_w4_quantize(W, group)
    q, s = _define(W, group)
    assert torch.equal(P.dequantize(), (q * s.float()[..., None]).view(n, k))
    # what pads the tiles: codes 8, scales 0
    nt, kt = P.words.shape[:2]
    full = binding.W4Weights(P.words, P.scales, nt * 16, kt * 128, group).dequantize()
    assert torch.count_nonzero(full[n:]) == 0 and torch.count_nonzero(full[:, k:]) == 0


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("n,k", [(1, 128), (24, 128), (40, 640), (2048, 2048), (17, 8064 + 128), (5632, 256), (333, 1152)])
def test_matvec(cuda_dev, n, k, N, group):
    P = binding.twell_w4_quantize(_weights(cuda_dev, n, k, 3 * n + k), group)
    g = torch.Generator("cpu").manual_seed(N)
    x = torch.randn((N, k), generator=g)
    x[:, ::37] *= 30
    x = x.to(BF).to(cuda_dev)
    y = binding.twell_w4_matvec(x, P)
    W = P.dequantize().double()
    ref = x.double() @ W.t()
    bound = 2.0 ** -8 * ref.abs() + k * 2.0 ** -22 * (x.double().abs() @ W.abs().t())
    err = (y.double() - ref).abs()
    assert (err <= bound).all(), (err / bound.clamp_min(1e-300)).max().item()
    assert torch.equal(y, binding.twell_w4_matvec(x, P))
    # a token's result does not depend on the others in the batch
    assert torch.equal(y[:1], binding.twell_w4_matvec(x[:1].contiguous(), P))


@pytest.mark.parametrize("k,group", [(32, 32), (96, 32), (192, 64), (160, 32)])
def test_columns_that_end_inside_a_tile(cuda_dev, k, group):
    P = binding.twell_w4_quantize(_weights(cuda_dev, 50, k, k), group)
    x = torch.randn((3, k), generator=torch.Generator("cpu").manual_seed(1)).to(BF).to(cuda_dev)
    ref = x.double() @ P.dequantize().double().t()
    y = binding.twell_w4_matvec(x, P).double()
    bound = 2.0 ** -8 * ref.abs() + k * 2.0 ** -22 * (x.double().abs() @ P.dequantize().double().abs().t())
    assert ((y - ref).abs() <= bound).all()


def test_integers_are_exact(cuda_dev):
    """Integer weights in -7..7 with a largest value of 7 have the scale 1; every sum is exact."""
    g = torch.Generator("cpu").manual_seed(4)
    W = torch.randint(-7, 8, (64, 512), generator=g).float()
    W[:, ::32] = 7
    x = torch.randint(-4, 5, (16, 512), generator=g).float()
    P = binding.twell_w4_quantize(W.to(BF).to(cuda_dev), 32)
    assert torch.equal(P.dequantize().cpu(), W)
    y = binding.twell_w4_matvec(x.to(BF).to(cuda_dev), P)
    assert torch.equal(y.cpu(), (x @ W.t()).to(BF))


def test_a_token_that_is_not_finite_stays_alone(cuda_dev):
    P = binding.twell_w4_quantize(_weights(cuda_dev, 48, 256, 9), 64)
    x = torch.randn((5, 256), generator=torch.Generator("cpu").manual_seed(2)).to(BF).to(cuda_dev)
    y = binding.twell_w4_matvec(x, P)
    x[2, 7] = float("nan")
    z = binding.twell_w4_matvec(x, P)
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], z[keep]) and torch.isnan(z[2]).all()


def test_weights_that_are_not_finite_are_reported(cuda_dev):
    W = _weights(cuda_dev, 16, 128, 10)
    W[3, 5] = float("inf")
    status = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    binding.twell_w4_quantize(W, 128, status=status)
    assert binding.twell_read_status(status) == 5


def test_refusals(cuda_dev):
    W = _weights(cuda_dev, 16, 128, 11)
    P = binding.twell_w4_quantize(W, 64)
    x = torch.zeros((17, 128), dtype=BF, device=cuda_dev)
    with pytest.raises(binding.TwellError) as e:
        binding.twell_w4_matvec(x, P)
    assert e.value.code == binding.TWELL_ERR_UNSUPPORTED
    for bad in (lambda: binding.twell_w4_matvec(x[:2, :64], P), lambda: binding.twell_w4_matvec(x[:2].float(), P),
                lambda: binding.twell_w4_quantize(W.float()), lambda: binding.twell_w4_quantize(W, 48),
                lambda: binding.twell_w4_quantize(W[:, :96].contiguous(), 64),
                lambda: binding.W4Weights(P.words, P.scales, 32, 128, 64),
                lambda: binding.W4Weights(P.words, P.scales, 16, 128, 32)):
        with pytest.raises(ValueError):
            bad()
    assert binding.twell_w4_matvec(x[:0], P).shape == (0, 16)


# Weights with more rows than two blocks an SM hold in two row tiles each, the last tile ragged: blocks of three and four row
# tiles, in one round and in several, with 7 and 8 warps.
@pytest.mark.parametrize("N", [1, 8, 9, 16])
@pytest.mark.parametrize("k,group", [(2560, 128), (4096, 32), (4128, 32), (1024, 64)])
@pytest.mark.parametrize("n", [9745, 14600, 24577])
def test_many_rows(cuda_dev, n, k, group, N):
    g = torch.Generator(cuda_dev).manual_seed(n + k)
    W = (torch.randn((n, k), generator=g, device=cuda_dev) / k ** 0.5).to(BF)
    P = binding.twell_w4_quantize(W, group)
    x = torch.randn((N, k), generator=g, device=cuda_dev).to(BF)
    y = binding.twell_w4_matvec(x, P)
    w = P.dequantize().double()
    ref = x.double() @ w.t()
    bound = 2.0 ** -8 * ref.abs() + k * 2.0 ** -22 * (x.double().abs() @ w.abs().t())
    err = (y.double() - ref).abs()
    assert (err <= bound).all(), (err / bound.clamp_min(1e-300)).max().item()
    assert torch.equal(y, binding.twell_w4_matvec(x, P))
    few = 1 if N <= 8 else 9  # the same bits in a smaller batch of the same kind
    assert torch.equal(y[:few], binding.twell_w4_matvec(x[:few].contiguous(), P))
