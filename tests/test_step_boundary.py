"""Host-side checks of the calls for a step's plan, rotation and adapters (no GPU): bad arguments are refused before
anything touches the device, and the frequencies are what their formulas say."""
import ctypes
import math
import os
import re
from fractions import Fraction

import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, build

INVALID, UNSUPPORTED, WORKSPACE, OK = 1, 2, 7, 0
A = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
BYTE = ctypes.c_void_p((1 << 20) + 1)
BF16, F32, E4M3 = binding.TWELL_BF16, binding.TWELL_F32, binding.TWELL_E4M3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _heads(**kw):
    f = dict(in_=1 << 20, out=1 << 21, n_heads=4, in_batch=4096, in_token=256, in_head=64, out_batch=4096, out_token=256, out_head=64)
    f.update(kw)
    return binding._RopeHeads(*f.values())


def _rope(lib, q=None, k=None, pos=A, pos_batch=0, turns=A, factor=1.0, B=1, S=8, hd=64, rot=64, nb=0, dt=BF16, bwd=False):
    fn = lib.twell_rope_bwd if bwd else lib.twell_rope_fwd
    ref = lambda h: None if h is None else ctypes.byref(h)  # noqa: E731
    return fn(ref(_heads() if q is None else q), ref(k), pos, pos_batch, turns, factor, B, S, hd, rot, nb, dt, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_rope_refuses(lib, bwd):
    for bad in (dict(pos=None), dict(turns=None), dict(B=-1), dict(S=-1), dict(hd=0), dict(rot=0), dict(rot=33), dict(rot=66),
                dict(nb=2), dict(nb=-1), dict(factor=0.0), dict(factor=-1.0), dict(factor=float("nan")), dict(factor=float("inf")),
                dict(pos=BYTE), dict(turns=ctypes.c_void_p((1 << 20) + 4)), dict(pos_batch=-8),
                dict(q=_heads(in_=None)), dict(q=_heads(out=None)), dict(q=_heads(n_heads=0)), dict(q=_heads(in_=(1 << 20) + 1)),
                dict(q=_heads(in_token=-256)), dict(k=_heads(n_heads=0)), dict(k=_heads(out=None)),
                # outputs that would lie over one another
                dict(q=_heads(out_token=0)), dict(q=_heads(out_head=32)), dict(q=_heads(out_token=200)), dict(B=3, q=_heads(out_batch=256)),
                dict(q=_heads(out_head=0)), dict(q=_heads(out_token=-256)),
                # in place with other strides
                dict(q=_heads(out=1 << 20, out_token=512))):
        assert _rope(lib, bwd=bwd, **bad) == INVALID, bad
    for bad in (dict(dt=E4M3), dict(dt=9), dict(hd=1032, rot=64), dict(S=1 << 25), dict(q=_heads(n_heads=65536, in_token=1 << 23, out_token=1 << 23))):
        assert _rope(lib, bwd=bwd, **bad) == UNSUPPORTED, bad
    assert _rope(lib, bwd=bwd, S=0, pos=None) == OK and _rope(lib, bwd=bwd, B=0, pos=None) == OK


def _plan(lib, n_pages=8, page=16, ring=1 << 20, state=1 << 20, table=A, mp=4, lens=A, news=1 << 22, labels=None, B=2, M=8, slots=A,
          pos=A, own=A, starts=A, lo=A, so=A, st=A):
    pool = binding._PagePool(n_pages, page, ring, state)
    return lib.twell_kv_plan(ctypes.byref(pool), table, mp, lens, news, labels, B, M, slots, pos, own, starts, lo, so, st, None)


def test_plan_refuses(lib):
    for bad in (dict(n_pages=-1), dict(page=0), dict(ring=None), dict(state=None), dict(table=None), dict(mp=0), dict(lens=None),
                dict(news=None), dict(B=-1), dict(M=-1), dict(slots=None), dict(pos=None), dict(own=None), dict(starts=None),
                dict(lo=None), dict(so=None), dict(st=None), dict(slots=ODD), dict(pos=ODD), dict(own=ODD), dict(lens=BYTE),
                dict(labels=BYTE), dict(table=BYTE), dict(state=(1 << 20) + 2), dict(lo=1 << 22), dict(labels=1 << 23, lo=1 << 23)):
        assert _plan(lib, **bad) == INVALID, bad
    for bad in (dict(page=12), dict(page=2048), dict(B=4097), dict(n_pages=1 << 27), dict(M=(1 << 31) - 1)):
        assert _plan(lib, **bad) == UNSUPPORTED, bad


X = ctypes.c_void_p(1 << 22)


def _lora(lib, y=A, ldy=64, x=X, ldx=128, L=2, R=16, k=128, n=64, a=1 << 20, b=1 << 20, scale=1 << 20, ranks=None, ids=A, N=4, out=A,
          ldo=64, ws=A, nb=1 << 30, st=A):
    ad = binding._Adapters(L, R, k, n, a, b, scale, ranks)
    return lib.twell_lora_add(y, ldy, x, ldx, ctypes.byref(ad), ids, N, out, ldo, ws, nb, st, None)


def test_lora_refuses(lib):
    for bad in (dict(y=None), dict(x=None), dict(a=None), dict(b=None), dict(scale=None), dict(ids=None), dict(out=None), dict(st=None),
                dict(N=-1), dict(L=0), dict(R=0), dict(k=0), dict(n=0), dict(R=12), dict(k=100), dict(n=60), dict(y=ODD, out=ODD),
                dict(x=ODD), dict(out=ODD), dict(a=(1 << 20) + 8), dict(b=(1 << 20) + 8), dict(scale=(1 << 20) + 2), dict(ids=BYTE),
                dict(ranks=(1 << 20) + 1), dict(ldy=60), dict(ldx=120), dict(ldx=132), dict(ldo=56), dict(ldo=72), dict(x=A)):
        assert _lora(lib, **bad) == INVALID, bad
    for bad in (dict(R=136), dict(L=4097), dict(N=(1 << 20) + 1), dict(k=(1 << 20) + 8, ldx=1 << 21), dict(n=(1 << 20) + 8, ldy=1 << 21, ldo=1 << 21)):
        assert _lora(lib, **bad) == UNSUPPORTED, bad
    assert _lora(lib, N=0, x=None) == OK


def test_lora_workspace(lib):
    ws = lambda N: lib.twell_workspace_bytes(binding.OP_LORA_ADD, N, 16, 1, 0, 0, 0)  # noqa: E731
    for N in (1, 64, 5000, 1 << 20):
        need = ws(N)
        assert ws(1 << 20) >= need >= ws(0)
        if need:
            for bad in (dict(ws=None), dict(ws=ODD), dict(nb=need - 1)):
                assert _lora(lib, N=N, **bad) == WORKSPACE, (N, bad)


def test_codes_match_the_header():
    src = open(os.path.join(build.INCLUDE, "twell.h")).read()
    assert int(re.search(r"TWELL_OP_LORA_ADD = (\d+)", src).group(1)) == binding.OP_LORA_ADD
    code = int(re.search(r"TWELL_ERR_POOL_EMPTY = (\d+)", src).group(1))
    assert binding.STATUS_NAMES[code] == "TWELL_ERR_POOL_EMPTY"
    assert binding._status_string(code) not in ("?", "unknown status")


def test_native_calls_refuse_before_the_device(lib):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    ints = torch.zeros(4, dtype=torch.int32)
    rot = binding.Rotary([1.0], 64, device="cpu")
    with pytest.raises(ValueError):
        binding.twell_rope_fwd(x, x, ints, rot)
    pool = binding.PagePool.full(8, 16, device="cpu")
    with pytest.raises(ValueError):
        binding.twell_kv_plan(pool, ints.view(4, 1), ints, ints, 4)
    ad = binding.Adapters(torch.zeros((2, 8, 64), dtype=torch.bfloat16), torch.zeros((2, 16, 8), dtype=torch.bfloat16), torch.zeros(2))
    with pytest.raises(ValueError):
        binding.twell_lora_add(x[:, 0, :16], x[:, 0], ad, ints)
    with pytest.raises(ValueError):
        binding._native.lora_add(x[:, 0, :16], x[:, 0], ad.a, ad.b, ad.scale, None, ints, x[:, 0, :16], None, ints, None)
    for name, count in (("rope", 11), ("kv_plan", 15), ("lora_add", 11)):
        with pytest.raises(TypeError):
            getattr(binding._native, name)(*[x] * (count - 1))


def test_rotary_lays_out_turns():
    for f in (1.0, 1e-4, 0.5, -0.25, 6.5, 2 * math.pi):
        t = int(binding.Rotary([f], 8, device="cpu").turns[0]) % 2 ** 64
        want = Fraction(f) / (2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")) * 2 ** 64 % 2 ** 64
        assert min(abs(t - want), 2 ** 64 - abs(t - want)) <= 1
    for bad in (dict(frequencies=[]), dict(frequencies=[1.0] * 5), dict(frequencies=[float("nan")]), dict(frequencies=[1.0], factor=0.0),
                dict(frequencies=[1.0], factor=float("inf"))):
        with pytest.raises(ValueError):
            binding.Rotary(head_dim=8, device="cpu", **bad)


def test_scaled_frequencies():
    f, m = binding.scaled_frequencies(8, 10000.0)
    assert m == 1.0 and all(math.isclose(a, b) for a, b in zip(f, (1.0, 0.1, 0.01, 0.001)))
    g, _ = binding.scaled_frequencies(8, 10000.0, "linear", 4.0)
    assert all(math.isclose(a, b / 4) for a, b in zip(g, f))
    g, _ = binding.scaled_frequencies(8, 10000.0, "base", 4.0)
    assert g[0] == 1.0 and math.isclose(g[3], f[3] / 4)
    f, _ = binding.scaled_frequencies(128, 500000.0)
    g, _ = binding.scaled_frequencies(128, 500000.0, "bands", 8.0, original=8192)
    for a, b in zip(f, g):
        turns = 8192 * a / (2 * math.pi)
        share = min(max((turns - 1) / 3, 0.0), 1.0)
        assert math.isclose(b, a * share + a / 8 * (1 - share), rel_tol=1e-12)
    assert g[0] == f[0] and math.isclose(g[-1], f[-1] / 8) and any(a / 8 < b < a for a, b in zip(f[1:], g[1:]))
    g, m = binding.scaled_frequencies(128, 10000.0, "ramp", 4.0, original=4096)
    f, _ = binding.scaled_frequencies(128, 10000.0)
    assert math.isclose(m, 0.1 * math.log(4) + 1) and g[0] == f[0] and math.isclose(g[-1], f[-1] / 4)
    ratio = [b / a for a, b in zip(f, g)]
    first = math.floor(128 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(10000.0)))
    last = math.ceil(128 * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000.0)))
    for i, r in enumerate(ratio):
        assert math.isclose(r, 1 - 0.75 * min(max((i - first) / (last - first), 0.0), 1.0), rel_tol=1e-12)
    assert binding.scaled_frequencies(2, 10000.0, "base", 4.0)[0] == [1.0]
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="bands", factor=2.0), dict(rot_dim=8, scaling="other"),
                dict(rot_dim=8, factor=0.5), dict(rot_dim=8, base=1.0), dict(rot_dim=8, scaling="ramp", factor=2.0),
                dict(rot_dim=8, scaling="bands", factor=2.0, original=64, low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            binding.scaled_frequencies(**bad)


def test_plans_and_pools_check_sizes(lib):
    pool = binding.PagePool.full(8, 16, device="cpu")
    assert pool.ring.tolist() == list(range(8)) and pool.state.tolist() == [0, 8, 0, 0]
    with pytest.raises(ValueError):
        binding.PagePool.full(-1, 16, device="cpu")
    ints = torch.zeros(4, dtype=torch.int32)
    plan = binding.StepPlan(ints, ints, ints, ints)
    with pytest.raises(ValueError):
        binding.twell_kv_plan(pool, ints.view(4, 1), ints, ints, 5, plan=plan)
    with pytest.raises(ValueError):
        binding.twell_kv_plan(pool, ints.view(4, 1), ints, ints, -1)
