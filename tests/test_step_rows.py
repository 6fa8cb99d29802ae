"""The rows of a step's tokens in the requests' page table and lengths (StepPlan.per_token), on the host."""
import random

import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding

I32 = torch.int32


@pytest.mark.parametrize("seed", range(8))
def test_rows_of_tokens(seed):
    r = random.Random(seed)
    B, cols = r.randint(1, 9), r.randint(1, 5)
    new = [r.choice([-1, 0, 0, 1, 1, 3]) for _ in range(B)]
    lens = [max(a, 0) + r.randint(0, 7) for a in new]
    served = [r.random() < 0.8 for _ in range(B)]
    starts, slots, want_rows, want_lens = [0], [], [], []
    table = torch.arange(B * cols, dtype=I32).view(B, cols)
    for b, a in enumerate(new):
        for i in range(max(a, 0)):
            slots.append(5 * b + i if served[b] else -1)
            want_rows.append(b)
            want_lens.append(lens[b] - max(a, 0) + i + 1 if served[b] else 0)
        starts.append(starts[-1] + max(a, 0))
    n, pad = len(slots), r.randint(0, 4)
    t = lambda v: torch.tensor(v, dtype=I32)  # noqa: E731
    plan = binding.StepPlan(t(slots + [-1] * pad), t([0] * (n + pad)), t([0] * (n + pad)), t(starts))
    rows, seen = plan.per_token(table, t(lens))
    assert rows.shape == (n + pad, cols) and rows.dtype == seen.dtype == I32
    assert torch.equal(rows[:n], table[want_rows]) and seen.tolist() == want_lens + [0] * pad


def test_no_requests_and_other_batches():
    e = torch.empty(0, dtype=I32)
    plan = binding.StepPlan(torch.full((3,), -1, dtype=I32), torch.zeros(3, dtype=I32), torch.full((3,), -1, dtype=I32), torch.zeros(1, dtype=I32))
    rows, seen = plan.per_token(torch.empty((0, 2), dtype=I32), e)
    assert rows.tolist() == [[0, 0]] * 3 and seen.tolist() == [0] * 3
    for table, lens in ((torch.zeros((1, 2), dtype=I32), torch.zeros(1, dtype=I32)), (torch.empty((0, 2), dtype=I32), torch.zeros(1, dtype=I32))):
        with pytest.raises(ValueError):
            plan.per_token(table, lens)
