"""The rotation, the plan and the adapters at sizes where their loops turn: several heads a warp, several tokens and pages a
thread, copies whose ring comes round, more tiles than the device holds at once. Bounds as in the operators' own tests."""
import pytest
import torch
from test_gpu_lora import _adapters, _check, _ids, _rand
from test_gpu_plan import _make, _run, _same, _walk
from test_gpu_rope import _angles
from test_gpu_rope import _check as _check_turned
from test_gpu_rope import _rand as _normal

from activation_sparse_ffn_gate_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()
    binding.status_buffer(cuda_dev).zero_()
    yield
    assert binding.twell_read_status() == 0, "device status was raised"


# a block's warps take every fourth head here: up to six a warp, and the keys go on where the queries end, at every remainder
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,hd,rot,hq,hk,interleaved", [(10007, 128, 128, 16, 8, False), (10001, 128, 64, 20, 4, True), (13003, 96, 96, 7, 3, False),
                                                        (9001, 128, 96, 5, 2, False), (20011, 80, 20, 9, 1, False), (8003, 64, 34, 6, 6, True),
                                                        (5003, 256, 256, 21, 0, False), (40009, 64, 64, 1, 9, False)])
def test_rotation_of_many_tokens(cuda_dev, N, hd, rot, hq, hk, interleaved, dtype):
    freq, factor = binding.scaled_frequencies(rot, 10000.0, "ramp", 4.0, original=4096)
    r = binding.Rotary(freq, hd, interleaved, factor)
    rows = _normal(cuda_dev, N, hq + 2 * hk, hd, seed=N, dtype=dtype)
    q, k = rows[:, :hq], rows[:, hq:hq + hk] if hk else None
    some = torch.randint(0, 100000, (61,), generator=torch.Generator().manual_seed(N), dtype=I32)
    which = torch.arange(N) * 7 % 61
    pos, angle = some[which].to(cuda_dev), _angles(some, freq)[which].to(cuda_dev)
    gq, gk = binding.twell_rope_fwd(q, k, pos, r)
    _check_turned(gq, q, angle, factor, interleaved)
    dq, dk = binding.twell_rope_bwd(q, k, pos, r)
    _check_turned(dq, q, angle, factor, interleaved, back=True)
    if hk:
        _check_turned(gk, k, angle, factor, interleaved)
        _check_turned(dk, k, angle, factor, interleaved, back=True)
    keep = rows.clone()
    binding.twell_rope_fwd(q, k, pos, r, q, k)  # in place, as the decoder layer calls it
    assert torch.equal(rows[:, :hq], gq) and (not hk or torch.equal(rows[:, hq:hq + hk], gk))
    assert torch.equal(rows[:, hq + hk:], keep[:, hq + hk:])


def test_rotation_of_a_training_batch(cuda_dev):
    B, S, hd, rot = 3, 4099, 128, 96
    freq, _ = binding.scaled_frequencies(rot)
    r = binding.Rotary(freq, hd)
    q, k = (_normal(cuda_dev, B, h, S, hd, seed=h).transpose(1, 2) for h in (10, 3))
    pos = torch.stack([(torch.arange(S, dtype=I32) + 11 * b) % 97 for b in range(B)])
    angle = _angles(torch.arange(97, dtype=I32), freq)[pos.long()].to(cuda_dev)
    gq, gk = binding.twell_rope_bwd(q, k, pos.to(cuda_dev), r, torch.empty_like(q), torch.empty_like(k))
    _check_turned(gq, q, angle, 1.0, False, back=True)
    _check_turned(gk, k, angle, 1.0, False, back=True)


# more tokens than 8 blocks an SM of 256 or 512 threads take at once, four each; pages of one token
@pytest.mark.parametrize("page,past,new", [(64, 300, [700_001, 650_000, 3, 701_003]), (1, 600_000, [400_001, 250_000, -1, 1, -1]),
                                           (16, 50, [4700 + 3 * (b % 17) for b in range(600)])])
def test_plans_of_more_tokens_than_threads(cuda_dev, page, past, new):
    at = iter(new)
    ring, state, table, lens, new = _make(page, len(new), page, past, lambda r: next(at))
    M = sum(max(a, 0) for a in new) + 5
    for in_place in (True, False):
        want = _walk(ring, state, page, table, lens, new, M)
        assert not want[8]
        _same(_run(cuda_dev, ring, state, page, table, lens, new, M, in_place=in_place), want)


def _both_ways(dev, N, k, n, R, L, form, ragged):
    ad = _adapters(dev, L, R, k, n, seed=N + R, ragged=ragged)
    ids = _ids(dev, N, L, N, form)
    x, y = _rand(dev, N, k, seed=N + 1), _rand(dev, N, n, seed=N + 2)
    out = binding.twell_lora_add(y, x, ad, ids, out=torch.full_like(y, 7.0))
    _check(out, y, x, ad, ids)
    assert torch.equal(binding.twell_lora_add(y, x, ad, ids), out)  # in place


# widths of 64 pieces and a rest, in a cluster, in two kernels, grouped: every ring comes round, its last slot half used
@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 128])
@pytest.mark.parametrize("N,L,form", [(1, 2, "one"), (40, 2, "any"), (40, 60, "any"), (700, 2, "runs"), (700, 40, "any"), (3001, 30, "runs"), (12000, 5, "runs")])
def test_adapters_of_wide_projections(cuda_dev, N, L, form, R):
    _both_ways(cuda_dev, N, 4104, 4104, R, L, form, ragged=R > 16)


@pytest.mark.parametrize("N,k,n,R", [(1, 16392, 12296, 16), (1, 9224, 16392, 64), (5, 20488, 264, 32), (9, 264, 30000, 128), (300, 14344, 72, 64),
                                     (300, 72, 14344, 16), (1500, 11272, 136, 24), (1500, 136, 11272, 64), (17000, 2056, 1032, 16)])
def test_adapters_of_long_and_short_sides(cuda_dev, N, k, n, R):
    _both_ways(cuda_dev, N, k, n, R, 3, "any", ragged=False)
