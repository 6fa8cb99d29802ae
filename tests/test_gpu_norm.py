"""GPU parity of the residual addition + RMS norm and its gradients (twell_add_rmsnorm_fwd / _bwd) against
the formulas in 64 bits.

Bounds, with u = 2^-24 (fp32) and b = 2^-8 (half a bf16 step, relative: 8 significant bits):
* h is one fp32 addition, rounded once: (b + 4u) |h|, or 4u |h| in fp32.
* y: the sum of squares is over 8 values a thread, 5 + 5 shuffles and one addition a chunk; its relative
  error is below 64u, rstd's half of that plus a few u, and two products follow: 64u |y|, plus b |y| in bf16.
* 8 bits: half an e4m3 step (2^-4 of the value, or 2^-10 under the smallest normal) times the scale, plus
  64u |y|; the scale within 64u.
* dx = s (g - xh c) + dh, c a mean of d products: 64u (s |g| + s |xh| mean|g xh| + |dx|), plus rounding.
* dw is a sum of N products: (N + 64) u sum|dy xh|.
"""
import numpy as np
import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U, B = 2.0 ** -24, 2.0 ** -8
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()


def _rand(dev, shape, dtype, seed, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).to(dev)


def _ref_fwd(x, res, w):
    h = x.double() + (res.double() if res is not None else 0.0)
    s = 1.0 / torch.sqrt(h.square().mean(-1) + EPS)
    return h, s, h * s[:, None] * w.double()


def _half(dt):
    return B if dt == BF else 0.0


def _within(got, ref, bound, what):
    d = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), what
    worst = (d - bound).max().item() if d.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:g} over its bound (largest error {d.max().item():g})"


SHAPES = [(1, 8), (1, 2048), (3, 64), (5, 136), (7, 256), (64, 1000), (33, 2560), (2, 8192), (3, 8200), (2, 16384),
          (600, 72)]


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (BF, None), (F32, None)])
@pytest.mark.parametrize("N,d", SHAPES)
def test_forward(cuda_dev, N, d, types):
    dt, rt = types
    x, w = _rand(cuda_dev, (N, d), dt, 1), _rand(cuda_dev, (d,), dt, 2)
    res = _rand(cuda_dev, (N, d), rt, 3, 4.0) if rt is not None else None
    y, h, rstd = binding.twell_add_rmsnorm_fwd(x, w, res, EPS, training=True)
    rh, rs, ry = _ref_fwd(x, res, w)
    if res is None:
        assert h is None
    else:
        assert h.dtype == rt
        _within(h, rh, (_half(rt) + 4 * U) * rh.abs(), "h")
    _within(rstd, rs, 64 * U * rs, "rstd")
    _within(y, ry, (_half(dt) + 64 * U) * ry.abs(), "y")
    y2, _, none = binding.twell_add_rmsnorm_fwd(x, w, res, EPS)
    assert none is None and torch.equal(y, y2)


def _check8(y8, ry, group):
    N, d = ry.shape
    width = group or d
    for j, lo in enumerate(range(0, d, width)):
        part = ry[:, lo:lo + width]
        a = part.abs().amax(1).clamp_min(2.0 ** -60)
        _within(y8.scale[:, j], a / 448, 64 * U * a / 448, "scale")
        s = (a / 448)[:, None]
        got = y8.values[:, lo:lo + width].double() * y8.scale[:, j].double()[:, None]
        _within(got, part, torch.maximum(2.0 ** -4 * part.abs(), 2.0 ** -10 * s) + 64 * U * part.abs() + 2.0 ** -20 * s,
                "8-bit rows")


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("N,d", SHAPES)
def test_forward_8bit(cuda_dev, N, d, group):
    x, w, res = _rand(cuda_dev, (N, d), BF, 4), _rand(cuda_dev, (d,), BF, 5), _rand(cuda_dev, (N, d), F32, 6)
    x[0, : d // 2] *= 50  # groups of different size
    y8, h, _ = binding.twell_add_rmsnorm_fwd_q8(x, w, res, EPS, group)
    rh, _, ry = _ref_fwd(x, res, w)
    _within(h, rh, 4 * U * rh.abs(), "h")
    _check8(y8, ry, group)
    # with a 16-bit output beside it: the same y as without the codes
    y = torch.empty_like(x)
    again, _, _ = binding.twell_add_rmsnorm_fwd_q8(x, w, res, EPS, group, y=y)
    assert torch.equal(again.values.view(torch.uint8), y8.values.view(torch.uint8))
    assert torch.equal(y, binding.twell_add_rmsnorm_fwd(x, w, res, EPS)[0])


def test_zero_rows_and_in_place(cuda_dev):
    x, w = _rand(cuda_dev, (9, 512), BF, 7), _rand(cuda_dev, (512,), BF, 8)
    x[4] = 0
    y8, _, _ = binding.twell_add_rmsnorm_fwd_q8(x, w, None, EPS)
    assert torch.count_nonzero(y8.values[4].float()) == 0
    assert y8.scale[4].item() == np.float32(2.0 ** -60) / np.float32(448)
    res = _rand(cuda_dev, (9, 512), BF, 9)
    y, h, _ = binding.twell_add_rmsnorm_fwd(x, w, res, EPS)
    x2, r2 = x.clone(), res.clone()
    yy, hh, _ = binding.twell_add_rmsnorm_fwd(x2, w, r2, EPS, y=x2, h=r2)
    assert yy is x2 and hh is r2 and torch.equal(yy, y) and torch.equal(hh, h)


def test_not_finite_rows_stay_alone(cuda_dev):
    """A row that holds an infinity or NaN does not touch the others."""
    x, w = _rand(cuda_dev, (12, 1000), F32, 10), _rand(cuda_dev, (1000,), F32, 11)
    y, _, _ = binding.twell_add_rmsnorm_fwd(x, w, None, EPS)
    bad = x.clone()
    bad[3, 17], bad[8, 0] = float("inf"), float("nan")
    yb, _, _ = binding.twell_add_rmsnorm_fwd(bad, w, None, EPS)
    keep = [i for i in range(12) if i not in (3, 8)]
    assert torch.equal(yb[keep], y[keep])
    assert torch.isnan(yb[8]).all() and torch.isnan(yb[3, 17])


def _ref_bwd(dy, h, w, rstd, dh):
    s = rstd.double()[:, None]
    xh, g = h.double() * s, dy.double() * w.double()
    c = (g * xh).mean(-1, keepdim=True)
    dx = s * (g - xh * c) + (dh.double() if dh is not None else 0.0)
    big = s * g.abs() + s * xh.abs() * (g * xh).abs().mean(-1, keepdim=True) + dx.abs() + \
        (dh.double().abs() if dh is not None else 0.0)
    return dx, big, (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("types", [(BF, BF, BF), (BF, F32, F32), (BF, F32, BF), (BF, BF, F32), (F32, F32, F32), (F32, F32, BF)])
@pytest.mark.parametrize("N,d", SHAPES + [(3000, 136), (2000, 2048)])
def test_backward(cuda_dev, N, d, types, with_dh):
    dt, rt, gt = types
    h, w = _rand(cuda_dev, (N, d), rt, 12, 2.0), _rand(cuda_dev, (d,), dt, 13)
    dy = _rand(cuda_dev, (N, d), gt, 14)
    dh = _rand(cuda_dev, (N, d), gt, 15) if with_dh else None
    rstd = (1.0 / torch.sqrt(h.double().square().mean(-1) + EPS)).float()
    dx, dw = binding.twell_add_rmsnorm_bwd(dy, h, w, rstd, dh)
    assert dx.dtype == gt and dw.dtype == F32
    rdx, big, rdw, sdw = _ref_bwd(dy, h, w, rstd, dh)
    _within(dx, rdx, _half(gt) * rdx.abs() + 64 * U * big, "dx")
    _within(dw, rdw, (N + 64) * U * sdw, "dw")
    dx2, dw2 = binding.twell_add_rmsnorm_bwd(dy, h, w, rstd, dh)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_backward_against_differences(cuda_dev):
    """Central differences, in 64 bits, of <y, dy> + <h, dh> in random directions of x and w. The step 1e-4
    leaves an error of about 1e-8 of the second-order terms (inputs of size 1); the fp32 gradients are within
    64u of their parts, so the directional derivatives agree to 1e-5 of the sum of |gradient x direction|."""
    N, d = 6, 72
    x, w = _rand(cuda_dev, (N, d), F32, 16), _rand(cuda_dev, (d,), F32, 17)
    dy, dh = _rand(cuda_dev, (N, d), F32, 18), _rand(cuda_dev, (N, d), F32, 19)
    _, _, rstd = binding.twell_add_rmsnorm_fwd(x, w, None, EPS, training=True)
    dx, dw = binding.twell_add_rmsnorm_bwd(dy, x, w, rstd, dh)

    def f(xx, ww):
        s = 1.0 / torch.sqrt(xx.square().mean(-1, keepdim=True) + EPS)
        return ((xx * s * ww) * dy.double()).sum() + (xx * dh.double()).sum()

    for seed in range(8):
        vx, vw = _rand(cuda_dev, (N, d), F32, 100 + seed).double(), _rand(cuda_dev, (d,), F32, 200 + seed).double()
        e = 1e-4
        num = (f(x.double() + e * vx, w.double() + e * vw) - f(x.double() - e * vx, w.double() - e * vw)) / (2 * e)
        ana = (dx.double() * vx).sum() + (dw.double() * vw).sum()
        size = (dx.double() * vx).abs().sum() + (dw.double() * vw).abs().sum()
        assert (num - ana).abs().item() <= 1e-5 * size.item()


def test_backward_in_place_and_empty(cuda_dev):
    h, w, dy = _rand(cuda_dev, (40, 512), F32, 20), _rand(cuda_dev, (512,), F32, 21), _rand(cuda_dev, (40, 512), F32, 22)
    rstd = torch.rsqrt(h.square().mean(-1) + EPS)
    dx, dw = binding.twell_add_rmsnorm_bwd(dy, h, w, rstd)
    buf = dy.clone()
    dx2, dw2 = binding.twell_add_rmsnorm_bwd(buf, h, w, rstd, dx=buf)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    dx0, dw0 = binding.twell_add_rmsnorm_bwd(dy[:0], h[:0], w, rstd[:0])
    assert dx0.shape == (0, 512) and torch.count_nonzero(dw0) == 0
    y0, _, _ = binding.twell_add_rmsnorm_fwd(h[:0], w)
    assert y0.shape == (0, 512)


def test_side_stream(cuda_dev):
    """On another stream than the current one: the result is there once that stream is done."""
    h, w, dy = _rand(cuda_dev, (700, 2048), F32, 23), _rand(cuda_dev, (2048,), F32, 24), _rand(cuda_dev, (700, 2048), F32, 25)
    _, _, rstd = binding.twell_add_rmsnorm_fwd(h, w, None, EPS, training=True)
    dx, dw = binding.twell_add_rmsnorm_bwd(dy, h, w, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    dx2, dw2 = binding.twell_add_rmsnorm_bwd(dy, h, w, rstd, stream=s)
    s.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_refusals(cuda_dev):
    x, w = _rand(cuda_dev, (4, 512), BF, 26), _rand(cuda_dev, (512,), BF, 27)
    res = _rand(cuda_dev, (4, 512), BF, 28)
    f = binding.twell_add_rmsnorm_fwd
    with pytest.raises(ValueError):
        f(x.t(), w)  # not contiguous
    with pytest.raises(ValueError):
        f(x, w[:256])
    with pytest.raises(ValueError):
        f(x, w.float())
    with pytest.raises(ValueError):
        f(x, w, res[:2])
    with pytest.raises(ValueError):
        f(x, w, h=res)  # an h without res
    with pytest.raises(ValueError):
        f(x.cpu(), w)
    with pytest.raises(binding.TwellError) as e:
        f(x.float(), w.float(), res)  # fp32 x with a bf16 residual stream
    assert e.value.code == binding.TWELL_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        f(x.half(), w.half())
    with pytest.raises(binding.TwellError) as e:
        binding.twell_add_rmsnorm_fwd_q8(x, w, group=64)
    assert e.value.code == binding.TWELL_ERR_UNSUPPORTED
    with pytest.raises(binding.TwellError):
        f(x[:, :508].contiguous(), w[:508].contiguous())  # d not a multiple of 8
    with pytest.raises(ValueError):
        binding.twell_add_rmsnorm_bwd(x, x, w, torch.ones(3, device=cuda_dev))
    with pytest.raises(ValueError):
        binding.twell_add_rmsnorm_bwd(x, x, w, torch.ones(4, device=cuda_dev), dh=x.float())


# More rows than the device holds at once, so that a block goes over several: a row's results are those of the row
# alone, bit for bit, and within the bounds of a row.
@pytest.mark.parametrize("rt", [BF, F32, None])
@pytest.mark.parametrize("N,d", [(40001, 8), (5003, 136), (3001, 1208), (2001, 4096), (701, 8192)])
def test_forward_many_rows(cuda_dev, N, d, rt):
    x, w = _rand(cuda_dev, (N, d), BF, 31), _rand(cuda_dev, (d,), BF, 32)
    res = _rand(cuda_dev, (N, d), rt, 33, 4.0) if rt is not None else None
    y, h, rstd = binding.twell_add_rmsnorm_fwd(x, w, res, EPS, training=True)
    y8, _, _ = binding.twell_add_rmsnorm_fwd_q8(x, w, res, EPS, 128)
    _, rs, ry = _ref_fwd(x, res, w)
    _within(rstd, rs, 64 * U * rs, "rstd")
    _within(y, ry, (_half(BF) + 64 * U) * ry.abs(), "y")
    for lo in (0, N // 2, N - 3):
        rows = slice(lo, lo + 3)
        part = None if res is None else res[rows]
        one, _, _ = binding.twell_add_rmsnorm_fwd(x[rows], w, part, EPS)
        assert torch.equal(one, y[rows])
        one8, _, _ = binding.twell_add_rmsnorm_fwd_q8(x[rows], w, part, EPS, 128)
        assert torch.equal(one8.values.view(torch.uint8), y8.values[rows].view(torch.uint8))
        assert torch.equal(one8.scale, y8.scale[rows])


# Batches that fill the device's threads, whose rows are spread over them otherwise than a few rows are: within the bounds
# of a row, and still the row's results alone, bit for bit.
@pytest.mark.parametrize("out", ["same", "whole", "groups"])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (BF, None)])
@pytest.mark.parametrize("N,d", [(9001, 288), (2600, 1000), (1300, 2560), (700, 4104), (400, 8192)])
def test_forward_wide_batches(cuda_dev, N, d, types, out):
    dt, rt = types
    x, w = _rand(cuda_dev, (N, d), dt, 41), _rand(cuda_dev, (d,), dt, 42)
    res = _rand(cuda_dev, (N, d), rt, 43, 4.0) if rt is not None else None
    rh, rs, ry = _ref_fwd(x, res, w)
    if out == "same":
        y, h, rstd = binding.twell_add_rmsnorm_fwd(x, w, res, EPS, training=True)
        _within(y, ry, (_half(dt) + 64 * U) * ry.abs(), "y")
        _within(rstd, rs, 64 * U * rs, "rstd")
        few = binding.twell_add_rmsnorm_fwd(x[-5:], w, None if res is None else res[-5:], EPS, training=True)
        assert torch.equal(few[0], y[-5:]) and torch.equal(few[2], rstd[-5:])
    else:
        group = 128 if out == "groups" else 0
        y8, h, _ = binding.twell_add_rmsnorm_fwd_q8(x, w, res, EPS, group)
        _check8(y8, ry, group)
        few, _, _ = binding.twell_add_rmsnorm_fwd_q8(x[-5:], w, None if res is None else res[-5:], EPS, group)
        assert torch.equal(few.values.view(torch.uint8), y8.values[-5:].view(torch.uint8))
        assert torch.equal(few.scale, y8.scale[-5:])
    if res is not None:
        _within(h, rh, (_half(rt) + 4 * U) * rh.abs(), "h")


@pytest.mark.parametrize("N,d", [(5, 136), (64, 1000), (33, 2560), (3, 8200)])
def test_backward_from_the_forwards_own_values(cuda_dev, N, d):
    """As training runs it: h rounded to bf16 and the rstd of the unrounded sum, against the gradients at that sum. Each
    entry of xh is off by B of itself, so the mean of g xh by B mean|g xh| and their product by twice that and B^2; dw by B
    sum|dy xh|: beside the bounds above."""
    x, w = _rand(cuda_dev, (N, d), BF, 51), _rand(cuda_dev, (d,), BF, 52)
    res, dy, dh = _rand(cuda_dev, (N, d), BF, 53, 4.0), _rand(cuda_dev, (N, d), F32, 54), _rand(cuda_dev, (N, d), F32, 55)
    _, h, rstd = binding.twell_add_rmsnorm_fwd(x, w, res, EPS, training=True)
    assert h.dtype == BF
    dx, dw = binding.twell_add_rmsnorm_bwd(dy, h, w, rstd, dh)
    rh, rs, _ = _ref_fwd(x, res, w)
    rdx, big, rdw, sdw = _ref_bwd(dy, rh, w, rs, dh)
    xh, g = rh * rs[:, None], dy.double() * w.double()
    more = rs[:, None] * xh.abs() * (g * xh).abs().mean(-1, keepdim=True) * (2 * B + B * B)
    _within(dx, rdx, 64 * U * big * (1 + B) + more, "dx")
    _within(dw, rdw, (B + (N + 64) * U * (1 + B)) * sdw, "dw")


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("N,d", [(3000, 136), (500, 2560), (7, 8200)])
def test_scales_are_the_quotient(cuda_dev, N, d, group):
    """scale = a / 448, the fp32 quotient of the largest magnitude (of y in fp32, as it is written beside the codes), and the
    codes those of y * (448 / a)."""
    x, w = _rand(cuda_dev, (N, d), F32, 61), _rand(cuda_dev, (d,), F32, 62)
    y = torch.empty_like(x)
    y8, _, _ = binding.twell_add_rmsnorm_fwd_q8(x, w, None, EPS, group, y=y)
    width = group or d
    for j, lo in enumerate(range(0, d, width)):
        part = y[:, lo:lo + width]
        a = part.abs().amax(1).clamp_min(2.0 ** -60)
        top = torch.full_like(a, 448.0)  # tensors on both sides: a division by a number may become a product
        assert torch.equal(y8.scale[:, j], a / top)
        codes = (part * (top / a)[:, None]).to(torch.float8_e4m3fn)
        assert torch.equal(y8.values[:, lo:lo + width].contiguous().view(torch.uint8), codes.view(torch.uint8))
