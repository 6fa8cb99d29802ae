"""GPU parity of the rotary positions (twell_rope_fwd, twell_rope_bwd) against the formula in 64 bits.

An angle is exact to 2^-33 of a turn and 2^-34 for the frequency's own rounding; its rest after the nearest quarter, at most
pi / 4, takes three roundings of fp32 (2^-24 each, relative), which is below 2^-22; the series and the factor add three
more of 2^-24 to the cosine and sine, the products and the sum three to each term: 2^-21 of factor (|a| + |b|) covers
them. Then one rounding to the output's type."""
import math
from fractions import Fraction

import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()


def _rand(dev, *shape, seed, dtype=F32):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(dev)


def _angles(pos, freq):
    """Radians [..., pairs] in 64 bits, from the exact fraction of a turn."""
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
    flat = []
    turns = [Fraction(f) / two_pi for f in freq]
    for p in pos.reshape(-1).tolist():
        flat += [float(p * t % 1) * 2 * math.pi for t in turns]
    return torch.tensor(flat, dtype=torch.float64, device=pos.device).view(*pos.shape, len(freq))


def _check(got, x, angle, factor, interleaved, back=False):
    """x, got [..., tokens, heads, hd]; angle [..., tokens, pairs]."""
    half = angle.shape[-1]
    rot = 2 * half
    c, s = (angle.cos() * factor)[..., None, :], ((-angle if back else angle).sin() * factor)[..., None, :]
    X = x.double()
    a, b = (X[..., 0:rot:2], X[..., 1:rot:2]) if interleaved else (X[..., :half], X[..., half:rot])
    u, v = a * c - b * s, a * s + b * c
    room = factor * 2.0 ** -21 * (a.abs() + b.abs())
    G = got.double()
    gu, gv = (G[..., 0:rot:2], G[..., 1:rot:2]) if interleaved else (G[..., :half], G[..., half:rot])
    for g, ref in ((gu, u), (gv, v)):
        bound = room + HALF_STEP[x.dtype] * (ref.abs() + room)
        assert ((g - ref).abs() <= bound).all(), ((g - ref).abs() / bound).max().item()
    assert torch.equal(got[..., rot:], x[..., rot:])


# head sizes, turned part, heads: whole, half, odd numbers of pairs, one pair
SHAPES = [(64, 64, 4, 2), (128, 128, 16, 8), (128, 64, 5, 1), (96, 96, 6, 2), (80, 20, 7, 7), (64, 2, 3, 1), (50, 34, 2, 3), (256, 96, 2, 1),
          (7, 6, 3, 2), (128, 126, 1, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N", [1, 3, 130])
@pytest.mark.parametrize("hd,rot,hq,hk", SHAPES)
def test_rows(cuda_dev, hd, rot, hq, hk, N, interleaved, dtype):
    freq, factor = binding.scaled_frequencies(rot, 10000.0, "ramp", 4.0, original=4096)
    r = binding.Rotary(freq, hd, interleaved, factor)
    rows = _rand(cuda_dev, N, hq + 2 * hk, hd, seed=hd + rot + N, dtype=dtype)
    q, k = rows[:, :hq], rows[:, hq:hq + hk]  # slices of a fused projection
    pos = torch.randint(0, 100000, (N,), generator=torch.Generator().manual_seed(N), dtype=torch.int32).to(cuda_dev)
    angle = _angles(pos, freq)
    gq, gk = binding.twell_rope_fwd(q, k, pos, r)
    _check(gq, q, angle, factor, interleaved)
    _check(gk, k, angle, factor, interleaved)
    dq, dk = binding.twell_rope_bwd(q, k, pos, r)
    _check(dq, q, angle, factor, interleaved, back=True)
    _check(dk, k, angle, factor, interleaved, back=True)
    # queries alone give the same bits, and so does a call in place, which leaves the values alone
    assert torch.equal(binding.twell_rope_fwd(q, None, pos, r)[0], gq)
    keep = rows.clone()
    binding.twell_rope_fwd(q, k, pos, r, q, k)
    assert torch.equal(rows[:, :hq], gq) and torch.equal(rows[:, hq:hq + hk], gk) and torch.equal(rows[:, hq + hk:], keep[:, hq + hk:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("own_positions", [False, True])
@pytest.mark.parametrize("B,S,hd,rot,hq,hk", [(3, 37, 64, 64, 4, 2), (2, 130, 128, 96, 6, 3), (4, 1, 64, 32, 2, 2), (1, 600, 80, 80, 2, 1)])
def test_head_first_batches(cuda_dev, B, S, hd, rot, hq, hk, own_positions, dtype):
    """[sequences, heads, tokens, head_dim] tensors seen token first, with a sequence's own positions or common ones."""
    freq, _ = binding.scaled_frequencies(rot)
    r = binding.Rotary(freq, hd)
    q, k = (_rand(cuda_dev, B, h, S, hd, seed=h + S, dtype=dtype).transpose(1, 2) for h in (hq, hk))
    pos = torch.arange(S, dtype=torch.int32, device=cuda_dev)
    if own_positions:
        pos = torch.stack([(pos + 5 * b) % 29 for b in range(B)]).to(torch.int32)
    angle = _angles(pos, freq).expand(B, S, rot // 2)
    q_out, k_out = torch.empty_like(q), torch.empty((B, S, hk, hd), dtype=dtype, device=cuda_dev)  # another layout of k's
    gq, gk = binding.twell_rope_fwd(q, k, pos, r, q_out, k_out)
    _check(gq, q, angle, 1.0, False)
    _check(gk, k, angle, 1.0, False)


@pytest.mark.parametrize("offset,stride", [(1, 65), (2, 70), (3, 64), (4, 68), (0, 66)])
def test_addresses_of_any_alignment(cuda_dev, offset, stride):
    """Heads that begin between 16-byte boundaries: the same bits as aligned ones give, and nothing beside them is written."""
    freq, _ = binding.scaled_frequencies(64)
    for dtype in (BF, F32):
        for interleaved in (False, True):
            r = binding.Rotary(freq, 64, interleaved)
            buf = _rand(cuda_dev, 9 * 2 * stride + 8, seed=offset, dtype=dtype)
            q = buf[offset:].as_strided((9, 2, 64), (2 * stride, stride, 1))
            pos = torch.arange(9, dtype=torch.int32, device=cuda_dev) * 1000
            want = binding.twell_rope_fwd(q.contiguous(), None, pos, r)[0]
            out = torch.full_like(buf, 7.0)
            at = out[offset:].as_strided((9, 2, 64), (2 * stride, stride, 1))
            assert torch.equal(binding.twell_rope_fwd(q, None, pos, r, at)[0], want)
            at.fill_(7.0)
            assert bool((out == 7.0).all())


def test_far_and_negative_positions(cuda_dev):
    freq = [1.0, 0.731, 1e-3, 1e-7, 5.9]
    r = binding.Rotary(freq, 10)
    pos = torch.tensor([0, 1, -1, 4095, 1_000_003, 2_000_000_011, 2 ** 31 - 1, -2 ** 31, -77], dtype=torch.int32, device=cuda_dev)
    x = _rand(cuda_dev, len(pos), 3, 10, seed=1)
    got, _ = binding.twell_rope_fwd(x, None, pos, r)
    _check(got, x, _angles(pos, freq), 1.0, False)
    assert torch.equal(got[0], x[0])  # position 0 turns nothing


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_is_the_gradient(cuda_dev, interleaved):
    """<out, d> is linear in x: its differences along unit directions, formed in 64 bits from the call's own outputs, are the
    backward's values; both are fp32, off by 2^-21 (|a| + |b|) and a rounding a term."""
    freq, factor = binding.scaled_frequencies(12, 10000.0, "ramp", 8.0, original=64)
    r = binding.Rotary(freq, 16, interleaved, factor)
    pos = torch.tensor([5, 900], dtype=torch.int32, device=cuda_dev)
    d = _rand(cuda_dev, 2, 1, 16, seed=2)
    back, _ = binding.twell_rope_bwd(d, None, pos, r)
    for j in range(16):
        x = torch.zeros((2, 1, 16), device=cuda_dev)
        x[:, 0, j] = 1.0
        out, _ = binding.twell_rope_fwd(x, None, pos, r)
        diff = (out.double() * d.double()).sum((1, 2))
        room = 2.0 ** -20 * factor * d.double().abs().sum((1, 2))
        assert ((back[:, 0, j].double() - diff).abs() <= room).all()
    # there and back is factor^2
    x = _rand(cuda_dev, 2, 3, 16, seed=3)
    y, _ = binding.twell_rope_fwd(x, None, pos, r)
    z, _ = binding.twell_rope_bwd(y, None, pos, r)
    assert (z[..., :12] - factor ** 2 * x[..., :12]).abs().max() <= 2.0 ** -18 * x.abs().max() * factor ** 2
    assert torch.equal(z[..., 12:], x[..., 12:])


def test_values_that_are_not_finite_stay_in_their_pair(cuda_dev):
    freq, _ = binding.scaled_frequencies(64)
    r = binding.Rotary(freq, 72)
    pos = torch.arange(4, dtype=torch.int32, device=cuda_dev) + 1
    x = _rand(cuda_dev, 4, 2, 72, seed=4, dtype=BF)
    want = binding.twell_rope_fwd(x, None, pos, r)[0]
    x[1, 0, 5], x[2, 1, 70] = float("nan"), float("inf")
    got = binding.twell_rope_fwd(x, None, pos, r)[0]
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[1, 0, 5] = touched[1, 0, 37] = touched[2, 1, 70] = True
    assert torch.equal(got[~touched], want[~touched])
    assert torch.isnan(got[1, 0, [5, 37]]).all() and got[2, 1, 70] == float("inf")


def test_expanded_inputs_and_empty_calls(cuda_dev):
    freq, _ = binding.scaled_frequencies(32)
    r = binding.Rotary(freq, 32)
    pos = torch.arange(6, dtype=torch.int32, device=cuda_dev)
    one = _rand(cuda_dev, 1, 1, 32, seed=5, dtype=BF)
    got = binding.twell_rope_fwd(one.expand(6, 4, 32), None, pos, r, torch.empty((6, 4, 32), dtype=BF, device=cuda_dev))[0]
    assert torch.equal(got, binding.twell_rope_fwd(one.expand(6, 4, 32).contiguous(), None, pos, r)[0])
    q = torch.empty((0, 4, 32), dtype=BF, device=cuda_dev)
    assert binding.twell_rope_fwd(q, q, pos[:0], r)[0].shape == (0, 4, 32)


def test_refusals(cuda_dev):
    freq, _ = binding.scaled_frequencies(32)
    r = binding.Rotary(freq, 32)
    q = torch.zeros((4, 2, 32), dtype=BF, device=cuda_dev)
    pos = torch.zeros(4, dtype=torch.int32, device=cuda_dev)
    for bad in (lambda: binding.twell_rope_fwd(q, q.float(), pos, r), lambda: binding.twell_rope_fwd(q, q[:3], pos, r),
                lambda: binding.twell_rope_fwd(q, None, pos[:3], r), lambda: binding.twell_rope_fwd(q, None, pos.long(), r),
                lambda: binding.twell_rope_fwd(q[..., :30], None, pos, r), lambda: binding.twell_rope_fwd(q[0], None, pos, r),
                lambda: binding.twell_rope_fwd(q, None, pos.cpu(), r), lambda: binding.twell_rope_fwd(q, None, pos, r, q.float()),
                lambda: binding.twell_rope_fwd(q, None, pos, r, q[:, :1]), lambda: binding.twell_rope_fwd(q, None, pos, r, None, q),
                lambda: binding.twell_rope_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), None, pos, r)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        binding.twell_rope_fwd(q.half(), None, pos, r)
    for bad in (lambda: binding.twell_rope_fwd(q, None, pos, r, q[:1].expand(4, 2, 32)),  # rows over one another
                lambda: binding.twell_rope_fwd(q, None, pos, r, q.view(2, 4, 32).transpose(0, 1)),  # in place, other strides
                lambda: (lambda o: binding.twell_rope_fwd(q, q, pos, r, o, o))(torch.empty_like(q))):  # one output for both
        with pytest.raises(binding.TwellError) as e:
            bad()
        assert e.value.code == 1
    assert binding.twell_read_status() == 0
