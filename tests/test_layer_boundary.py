"""Host-side checks of the operators around the FFN (no GPU): bad arguments are refused before anything
touches the device, and the sizes are what the header says."""
import ctypes

import pytest

from activation_sparse_ffn_gate_gb300 import binding, build

INVALID, UNSUPPORTED, WORKSPACE, OK = 1, 2, 7, 0
A = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
BF16, F32, E4M3 = binding.TWELL_BF16, binding.TWELL_F32, binding.TWELL_E4M3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _fwd(lib, x=A, res=A, w=A, N=4, d=64, eps=1e-6, dt=BF16, rt=BF16, h=A, y=A, y8=None, sc=None, group=0, rstd=None):
    return lib.twell_add_rmsnorm_fwd(x, res, w, N, d, eps, dt, rt, h, y, y8, sc, group, rstd, None)


def test_rmsnorm_fwd_refuses(lib):
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(d=60), dict(d=0), dict(N=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(y8=A), dict(x=ODD), dict(res=ODD), dict(w=ODD), dict(h=ODD), dict(y=ODD),
                dict(y8=ODD, sc=A), dict(y8=A, sc=ODD), dict(rstd=ODD)):
        assert _fwd(lib, **bad) == INVALID, bad
    for bad in (dict(dt=F32, rt=BF16), dict(dt=E4M3), dict(dt=7), dict(rt=E4M3), dict(d=16392), dict(y8=A, sc=A, group=64)):
        assert _fwd(lib, **bad) == UNSUPPORTED, bad
    assert _fwd(lib, N=0, x=None, y=None) == OK


def _bwd(lib, dy=A, h=A, w=A, rstd=A, dh=None, N=4, d=64, dt=BF16, rt=F32, gt=F32, dx=A, dw=A, ws=A, ws_bytes=1 << 30):
    return lib.twell_add_rmsnorm_bwd(dy, h, w, rstd, dh, N, d, dt, rt, gt, dx, dw, ws, ws_bytes, None)


def test_rmsnorm_bwd_refuses(lib):
    for bad in (dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(dw=None), dict(d=12),
                dict(N=-1), dict(dy=ODD), dict(h=ODD), dict(w=ODD), dict(rstd=ODD), dict(dh=ODD), dict(dx=ODD), dict(dw=ODD)):
        assert _bwd(lib, **bad) == INVALID, bad
    for bad in (dict(dt=F32, rt=BF16), dict(gt=E4M3), dict(gt=7), dict(d=16392)):
        assert _bwd(lib, **bad) == UNSUPPORTED, bad
    need = lib.twell_workspace_bytes(binding.OP_ADD_RMSNORM_BWD, 4, 64, 1, 0, 0, 0)
    assert need > 0
    for bad in (dict(ws=None), dict(ws=ODD), dict(ws_bytes=need - 1)):
        assert _bwd(lib, **bad) == WORKSPACE, bad


def _cache(**kw):
    f = dict(n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, dtype=BF16, k=1 << 20, v=1 << 20, k_scale=None, v_scale=None,
             page_stride=2048, head_stride=1024, token_stride=64, scale_page_stride=32, scale_head_stride=16)
    f.update(kw)
    return binding._KVCache(*f.values())


BAD_CACHES = [dict(n_pages=-1), dict(page_size=0), dict(n_kv_heads=0), dict(head_dim=0), dict(k=None), dict(v=None),
              dict(k=(1 << 20) + 8), dict(token_stride=32), dict(token_stride=68), dict(head_stride=-1024), dict(page_stride=2044),
              dict(dtype=E4M3), dict(dtype=E4M3, k_scale=4096, v_scale=4096, page_stride=2056),
              dict(dtype=E4M3, k_scale=4096, v_scale=4096, scale_head_stride=-1)]
OTHER_CACHES = [dict(page_size=12), dict(page_size=2048), dict(head_dim=72), dict(head_dim=512, token_stride=512), dict(dtype=F32),
                dict(n_pages=1 << 28)]


@pytest.mark.parametrize("call", ["append", "gather", "attn"])
def test_cache_descriptor_is_checked(lib, call):
    def run(c):
        c = ctypes.byref(c)
        if call == "append":
            return lib.twell_kv_append(c, A, A, 128, 128, A, 1, A, None)
        if call == "gather":
            return lib.twell_kv_gather(c, A, 1, A, A, A, None)
        return lib.twell_paged_attn_decode(A, 256, c, A, A, 1, 4, 1, 1.0, 0, A, None, A, 1 << 30, A, None)

    for kw in BAD_CACHES:
        assert run(_cache(**kw)) == INVALID, kw
    for kw in OTHER_CACHES:
        assert run(_cache(**kw)) == UNSUPPORTED, kw


def test_append_and_gather_refuse(lib):
    c = ctypes.byref(_cache())
    ap = lambda k=A, v=A, ldk=128, ldv=128, s=A, n=1, st=A: lib.twell_kv_append(c, k, v, ldk, ldv, s, n, st, None)  # noqa: E731
    for bad in (dict(k=None), dict(v=None), dict(s=None), dict(st=None), dict(n=-1), dict(k=ODD), dict(v=ODD), dict(ldk=120),
                dict(ldv=132)):
        assert ap(**bad) == INVALID, bad
    assert ap(n=1 << 30) == UNSUPPORTED
    assert ap(n=0, k=None) == OK
    ga = lambda s=A, n=1, k=A, v=A, st=A: lib.twell_kv_gather(c, s, n, k, v, st, None)  # noqa: E731
    for bad in (dict(s=None), dict(k=None), dict(v=None), dict(st=None), dict(n=-1), dict(k=ODD), dict(v=ODD)):
        assert ga(**bad) == INVALID, bad
    assert ga(n=1 << 30) == UNSUPPORTED
    assert ga(n=0, k=None) == OK


def test_attention_refuses(lib):
    c = _cache()
    need = lib.twell_workspace_bytes(binding.OP_PAGED_ATTN, 2, 64, 1, 0, 0, 0)

    def f(q=A, qs=256, cache=c, table=A, lens=A, B=2, nq=4, mp=8, window=0, out=A, lse=None, ws=A, nb=need, st=A):
        return lib.twell_paged_attn_decode(q, qs, ctypes.byref(cache), table, lens, B, nq, mp, 1.0, window, out, lse, ws, nb, st,
                                           None)

    for bad in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(st=None), dict(B=-1), dict(nq=0), dict(nq=3),
                dict(mp=0), dict(window=-1), dict(q=ODD), dict(out=ODD), dict(lse=ODD), dict(qs=255), dict(qs=128)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(cache=_cache(head_dim=80, token_stride=80)), dict(B=4097), dict(mp=1 << 27), dict(B=4096, mp=1 << 20),
                dict(nq=65536, qs=65536 * 64)):
        assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=ODD), dict(nb=need - 1)):
        assert f(**bad) == WORKSPACE, bad
    assert f(B=0, q=None) == OK


def test_w4_refuses(lib):
    q = lambda W=A, n=16, k=128, g=64, w=A, s=A, st=A: lib.twell_w4_quantize(W, n, k, g, w, s, st, None)  # noqa: E731
    for bad in (dict(W=None), dict(w=None), dict(s=None), dict(st=None), dict(n=0), dict(k=0), dict(k=96), dict(g=0), dict(k=40, g=8),
                dict(W=ODD), dict(w=ODD), dict(s=ODD)):
        assert q(**bad) == INVALID, bad
    assert q(k=256, g=256) == UNSUPPORTED
    m = lambda x=A, w=A, s=A, N=1, n=16, k=128, g=64, y=A: lib.twell_w4_matvec(x, w, s, N, n, k, g, y, None)  # noqa: E731
    for bad in (dict(x=None), dict(w=None), dict(s=None), dict(y=None), dict(N=-1), dict(n=0), dict(k=0), dict(k=96), dict(x=ODD),
                dict(w=ODD), dict(s=ODD), dict(y=ODD)):
        assert m(**bad) == INVALID, bad
    for bad in (dict(N=17), dict(k=256, g=256), dict(n=(1 << 24) + 1), dict(k=(1 << 24) + 128)):
        assert m(**bad) == UNSUPPORTED, bad
    assert q(n=(1 << 24) + 1) == UNSUPPORTED
    assert m(N=0, x=None) == OK


def test_sizes(lib):
    assert lib.twell_w4_words_bytes(16, 128) == 1024
    assert lib.twell_w4_words_bytes(17, 160) == 4 * 1024
    assert lib.twell_w4_words_bytes(0, 128) == 0
    assert lib.twell_w4_scales_bytes(17, 160, 32) == 4 * 16 * 4 * 2
    assert lib.twell_w4_scales_bytes(16, 128, 128) == 32
    assert lib.twell_w4_scales_bytes(16, 128, 100) == 0
    ws = lambda op, N, d: lib.twell_workspace_bytes(op, N, d, 1, 0, 0, 0)  # noqa: E731
    assert ws(binding.OP_ADD_RMSNORM_BWD, 0, 64) == 0 and ws(binding.OP_ADD_RMSNORM_BWD, 4, 60) == 0
    assert ws(binding.OP_ADD_RMSNORM_BWD, 5000, 2048) >= ws(binding.OP_ADD_RMSNORM_BWD, 50, 2048) > 0
    assert ws(binding.OP_PAGED_ATTN, 0, 64) == 0
    assert ws(binding.OP_PAGED_ATTN, 64, 128) > ws(binding.OP_PAGED_ATTN, 64, 64) > 0


def test_enums_match_the_header():
    import os
    import re
    src = open(os.path.join(build.INCLUDE, "twell.h")).read()
    for name in ("TWELL_OP_ADD_RMSNORM_BWD", "TWELL_OP_PAGED_ATTN"):
        assert int(re.search(name + r" = (\d+)", src).group(1)) == getattr(binding, name[len("TWELL_"):])
    assert int(re.search(r"TWELL_E4M3 = (\d+)", src).group(1)) == binding.TWELL_E4M3


def test_native_calls_refuse_before_the_device(lib):
    """The native module checks what it is given: no tensor, a tensor on the host, another number of arguments."""
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.twell_add_rmsnorm_fwd(x, x[0])
    with pytest.raises(TypeError):
        binding._native.add_rmsnorm_fwd(x, x[0])
    with pytest.raises(TypeError):
        binding._native.w4_matvec(1, x, x, 16, 128, 64, x, None)
    with pytest.raises(ValueError):
        binding._native.w4_matvec(x, x, x, 16, 128, 64, x, None)


def test_missing_native_calls_are_not_passed_over(lib, monkeypatch):
    """Without the native module load() raises: there is no slower way around it."""
    import importlib

    def missing(name, package=None):
        raise ImportError(name)

    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(importlib, "import_module", missing)
    with pytest.raises(RuntimeError):
        binding.load()


def test_attention_refuses_lengths_near_32_bits(lib):
    """A length is rounded up to a tile of 32 tokens in 32 bits: tables whose length would not survive that are refused."""
    need = lib.twell_workspace_bytes(binding.OP_PAGED_ATTN, 1, 64, 1, 0, 0, 0)
    for ps, mp in ((1, (1 << 31) - 20), (1, (1 << 31) - 31), (8, (1 << 28) - 3), (1, (1 << 31) - 17)):
        c = _cache(page_size=ps, page_stride=2 * 64 * ps, head_stride=64 * ps)
        st = lib.twell_paged_attn_decode(A, 256, ctypes.byref(c), A, A, 1, 4, mp, 1.0, 0, A, None, A, need, A, None)
        assert st == UNSUPPORTED, (ps, mp)


def test_the_ffn_runs_without_the_native_calls(lib, monkeypatch):
    """Its calls go through ctypes and need the library alone."""
    import importlib

    def missing(name, package=None):
        raise ImportError(name)

    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_native", None)
    monkeypatch.setattr(importlib, "import_module", missing)
    assert binding.twell_workspace_bytes(binding.OP_FFN_FUSED_FWD, 64, 512, 1024) > 0
    with pytest.raises(RuntimeError):
        binding.load()


def test_native_calls_are_built_again_for_another_torch(lib, monkeypatch):
    import torch
    assert build._stale() == (False, False)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert build._stale() == (False, True)


def test_a_library_from_elsewhere(lib, monkeypatch, tmp_path):
    """load(path) takes a library that lies elsewhere, without native calls beside it."""
    import importlib
    import shutil

    def missing(name, package=None):
        raise ImportError(name)

    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_native", None)
    monkeypatch.setattr(importlib, "import_module", missing)
    path = str(shutil.copy(binding.LIB_PATH, tmp_path / "elsewhere.so"))
    other = binding.load(path)
    assert other._name == path and other.twell_workspace_bytes(binding.OP_FFN_FUSED_FWD, 64, 512, 1024, 8, 0, 0) > 0
    with pytest.raises(RuntimeError):
        binding.twell_add_rmsnorm_fwd(None, None, y=1)
