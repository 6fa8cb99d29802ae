"""Waits of the adapters' kernels that run out, without a fault or a hang: in a process whose limit is a nanosecond, a block gives up
on sums that the others of its cluster are about to send. It stays until they have come, records TWELL_ERR_TIMEOUT, and what
would need those sums is not written: its own columns, or the rows whose t it had to put together.

Small integers: every sum is exact, so that an output is the formula's or untouched, to the bit."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

pytestmark = pytest.mark.gpu
TIMEOUT = 4


def _case(N, L, R, k, n):
    """x with four values of 1 a row, a with 1 and 2 in four of its ranks, b with ones: 0 < b t <= 32, and y between -64 and -8."""
    g = torch.Generator().manual_seed(N + R)
    x = torch.zeros((N, k)).scatter_(1, torch.randint(0, k, (N, 4), generator=g), 1.0)
    a = torch.randint(1, 3, (L, R, k), generator=g).float()
    a[:, 4:] = 0
    b = torch.ones((L, n, R))
    y = 8.0 * torch.randint(-8, 0, (N, n), generator=g)
    ids = torch.randint(0, L, (N,), generator=g)
    want = y + torch.einsum("mr,mnr->mn", torch.einsum("mrk,mk->mr", a[ids], x), b[ids[:, None], torch.arange(n)])
    assert want.abs().max() <= 64 and (want != y).all()
    return [t.cuda() for t in (x.bfloat16(), a.bfloat16(), b.bfloat16(), y.bfloat16(), ids.int(), want.bfloat16())]


def _child():
    from activation_sparse_ffn_gate_gb300 import binding
    gave_up = []
    # one kernel, a cluster of eight blocks a tile; then tokens grouped first, eight blocks and fewer a tile in the first product
    for N, L, R, k, n in ((1, 2, 16, 1024, 1032), (3, 2, 64, 512, 520), (40, 2, 128, 520, 264), (1100, 2, 16, 1024, 264), (2100, 3, 40, 264, 136)):
        x, a, b, y, ids, want = _case(N, L, R, k, n)
        ad = binding.Adapters(a, b, torch.ones(L, device="cuda"))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(binding.twell_workspace_bytes(binding.OP_LORA_ADD, N, R, 1), dtype=torch.uint8, device="cuda")
        gave_up.append(0)
        for i in range(60):
            out = y.clone()
            ws.fill_(127)  # what no call has written is 3.4e38
            binding.twell_lora_add(out, x, ad, ids, ws=ws, status=status)
            code = binding.twell_read_status(status)
            assert code in (0, TIMEOUT), code
            gave_up[-1] += code == TIMEOUT
            assert ((out == y) | (out == want)).all(), (N, i)
            if N > 512:  # a tile's rows together
                assert ((out == y).all(1) | (out == want).all(1)).all(), (N, i)
            if code == 0:
                assert torch.equal(out, want), (N, i)
    torch.cuda.synchronize()
    print("gave up", *gave_up)


def test_waits_that_run_out(cuda_dev):
    from activation_sparse_ffn_gate_gb300 import build
    build.build()
    run = subprocess.run([sys.executable, os.path.abspath(__file__)], env={**os.environ, "TWELL_WAIT_LIMIT_MS": "0.000001"}, cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout + run.stderr
    counts = [int(v) for v in run.stdout.split("gave up")[1].split()]
    print(counts)
    assert sum(counts[:3]) > 0 and sum(counts[3:]) > 0  # in one kernel, and after the tokens are grouped


if __name__ == "__main__":
    _child()
