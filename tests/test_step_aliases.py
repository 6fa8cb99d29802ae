"""Arguments of a step's calls that lie over one another are refused before anything touches the device (no GPU)."""
import pytest
import torch
from test_step_boundary import INVALID, _heads, _rope

from activation_sparse_ffn_gate_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("bwd", [False, True])
def test_an_output_over_the_other_sides_input(lib, bwd):
    """Blocks of one side would read what those of the other have turned already."""
    q, k = 1 << 20, 1 << 24
    for q_to, k_to in ((k, q), (k, 1 << 25), (1 << 25, q)):
        assert _rope(lib, q=_heads(in_=q, out=q_to), k=_heads(in_=k, out=k_to), bwd=bwd) == INVALID
    # the queries are the keys, and one of the two works in place
    assert _rope(lib, q=_heads(in_=q, out=q), k=_heads(in_=q, out=k), bwd=bwd) == INVALID
    assert _rope(lib, q=_heads(in_=q, out=k), k=_heads(in_=q, out=q), bwd=bwd) == INVALID


@pytest.mark.gpu
def test_swapped_outputs_are_refused(cuda_dev, lib):
    q, k = (torch.randn((5, 2, 64), device=cuda_dev) for _ in range(2))
    keep = q.clone(), k.clone()
    r, pos = binding.Rotary([1.0] * 32, 64), torch.arange(5, dtype=torch.int32, device=cuda_dev)
    for call in (lambda: binding.twell_rope_fwd(q, k, pos, r, k, q), lambda: binding.twell_rope_bwd(q, q, pos, r, q)):
        with pytest.raises(binding.TwellError) as e:
            call()
        assert e.value.code == INVALID
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])
