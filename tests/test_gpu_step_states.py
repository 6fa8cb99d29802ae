"""Steps of a served life that are not one new token for each request, and a pool whose state is lost."""
import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EMPTY, CHECK = 8, 5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()
    binding.status_buffer(cuda_dev).zero_()
    yield
    assert binding.twell_read_status() == 0, "device status was raised"


@pytest.mark.parametrize("state", [[9, 1, 0, 0], [-1, 3, 0, 0], [2, -1, 0, 0], [0, 9, 0, 0]])
def test_a_state_outside_the_ring_begins_an_empty_one(cuda_dev, state):
    """No page is taken; those of a request that has ended are all that the pool has from then on, and later steps take them."""
    t = lambda v: torch.tensor(v, dtype=I32, device=cuda_dev)  # noqa: E731
    pool = binding.PagePool(t([7, 6, 5, 4, 3, 2, 1, 0]), t(state), 4)
    table, lens, status = t([[3, 6, -1], [1, -1, -1], [5, -1, -1]]), t([7, 4, 2]), t([0])
    p = binding.twell_kv_plan(pool, table, lens, t([-1, 1, 1]), 2, status=status)
    assert binding.twell_read_status(status) == CHECK
    assert lens.tolist() == [0, 4, 3] and p.slots.tolist() == [-1, 22] and p.positions.tolist() == [0, 2]
    assert pool.state.tolist() == [0, 2, 0, 0] and pool.ring.tolist() == [3, 6, 5, 4, 3, 2, 1, 0]
    p = binding.twell_kv_plan(pool, table, lens, t([0, 1, 1]), 2, status=status)
    assert binding.twell_read_status(status) == 0
    assert p.slots.tolist() == [12, 23] and table[1].tolist() == [1, 3, -1] and pool.state.tolist() == [1, 1, 0, 0]
