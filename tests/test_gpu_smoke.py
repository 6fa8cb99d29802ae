"""The smoke run reaches every operator of the library's layers."""
import pytest

from activation_sparse_ffn_gate_gb300 import binding

pytestmark = pytest.mark.gpu


def test_smoke_runs_the_operators_around_the_ffn(cuda_dev, monkeypatch):
    import __graft_entry__
    seen = set()

    def watched(name, fn):
        def call(*args, **kwargs):
            seen.add(name)
            return fn(*args, **kwargs)
        return call

    names = ("twell_add_rmsnorm_fwd", "twell_add_rmsnorm_fwd_q8", "twell_add_rmsnorm_bwd", "twell_kv_append", "twell_kv_gather",
             "twell_paged_attn_decode", "twell_w4_quantize", "twell_w4_matvec")
    for name in names:
        monkeypatch.setattr(binding, name, watched(name, getattr(binding, name)))
    __graft_entry__.smoke()
    assert seen == set(names)
