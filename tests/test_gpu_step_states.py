"""Steps of a served life that are not one new token for each request, and a pool whose state is lost."""
import math

import pytest
import torch
from test_gpu_block import REL, _norm, _rand, _rel
from test_gpu_step import _adapted, _served, _turn

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


# new tokens of five requests: one that idles, one that has ended, a row that a prompt fills again, several tokens of one; with
# rows of padding up to five or more, as a captured step of a fixed size has them
STEPS = [[3, 1, 2, 1, 4], [1, 0, 1, 1, 1], [1, 1, -1, 0, 1], [0, 1, 0, 1, 1], [1, 0, 5, 1, 0], [-1, 1, 1, 2, 1], [0, 0, 0, 0, 0], [2, 1, 1, 1, 1]]


@pytest.mark.parametrize("window", [0, 5])
@pytest.mark.parametrize("cache_dtype", [BF, torch.float8_e4m3fn])
def test_a_token_sees_its_own_request(cuda_dev, cache_dtype, window):
    """Each token against the layer in 64 bits over its request's tokens up to it, by the bound of the served life's own test;
    padding rows see nothing."""
    d, hq, hk, hd, B, page, cols = 512, 8, 2, 64, 5, 4, 12
    layer, freq, factor = _served(cuda_dev, d, 1024, hq, hk, hd)
    pool = binding.PagePool.full(B * cols, page, cuda_dev)
    cache = binding.KVCache.empty(B * cols, page, hk, hd, cache_dtype, cuda_dev)
    table, lens = torch.full((B, cols), -1, dtype=I32, device=cuda_dev), torch.zeros(B, dtype=I32, device=cuda_dev)
    labels = torch.tensor([0, 2, -1, 1, 0], dtype=I32, device=cuda_dev)
    W, Wo = layer.w_qkv.dequantize().double(), layer.w_out.dequantize().double()
    have = [0] * B
    for step, new in enumerate(STEPS):
        rows = [(b, i) for b, n in enumerate(new) for i in range(n)]  # request, its new token's number
        n = max(B, len(rows))
        p = binding.twell_kv_plan(pool, table, lens, torch.tensor(new, dtype=I32, device=cuda_dev), n, labels=labels)
        t, seen = p.per_token(table, lens)
        upto = [have[b] + i + 1 for b, i in rows]
        assert seen.dtype == I32 and seen.tolist() == upto + [0] * (n - len(rows))
        assert torch.equal(t[:len(rows)], table[[b for b, _ in rows]])
        have = [0 if a < 0 else h + a for h, a in zip(have, new)]
        assert lens.tolist() == have
        delta, h = _rand(cuda_dev, n, d, seed=60 + step), _rand(cuda_dev, n, d, seed=80 + step, dtype=F32)
        out, h2 = layer.decode(delta, h, cache, p.slots, t, seen, window=window, positions=p.positions, adapter_ids=p.owner)
        h1 = delta.double() + h.double()
        y = _norm(h1, layer.attn_norm, layer.eps)
        qkv = (y @ W.t() + _adapted(y, layer.adapters_qkv, p.owner)).view(n, hq + 2 * hk, hd)
        q = _turn(qkv[:, :hq], p.positions, freq, factor).view(n, hk, hq // hk, hd)
        a = torch.zeros((n, hk, hq // hk, hd), dtype=torch.float64, device=cuda_dev)
        for row, (b, _) in enumerate(rows):
            at = torch.arange(max(0, upto[row] - window) if window else 0, upto[row], device=cuda_dev)
            k, v = binding.twell_kv_gather(cache, (table[b, at // page] * page + at % page).to(I32))
            z = torch.einsum("hgd,nhd->hgn", q[row], k.double()) / math.sqrt(hd)
            a[row] = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), v.double())
        a = a.view(n, hq * hd)
        r2 = h1 + a @ Wo.t() + _adapted(a, layer.adapters_out, p.owner)
        y = _norm(r2, layer.ffn_norm, layer.eps)
        ref = (torch.relu(y @ layer.Wg_s.double().t()) * (y @ layer.Wu_s.double().t())) @ layer.Wd_s.double()
        assert _rel(h2, r2) <= REL and _rel(out, ref) <= REL
        for row in range(n):  # none is far off alone: nine roundings of at most 2^-8 of their size are 0.035
            assert _rel(h2[row], r2[row]) <= 4 * REL


def test_a_request_without_pages_sees_nothing(cuda_dev):
    t = lambda v: torch.tensor(v, dtype=I32, device=cuda_dev)  # noqa: E731
    pool = binding.PagePool(t([0, 1]), t([0, 1, 0, 0]), 4)
    table, lens, status = t([[1, -1], [-1, -1], [-1, -1]]), t([3, 0, 0]), t([0])
    p = binding.twell_kv_plan(pool, table, lens, t([1, 2, 1]), 6, status=status)
    assert binding.twell_read_status(status) == EMPTY
    rows, seen = p.per_token(table, lens)
    assert seen.tolist() == [4, 1, 2, 0, 0, 0] and rows[:3].tolist() == table[[0, 1, 1]].tolist()
    with pytest.raises(ValueError):
        p.per_token(table[:2], lens[:2])
    with pytest.raises(ValueError):
        p.per_token(table, lens[:2])


def test_a_captured_step_takes_other_requests_in_its_replays(cuda_dev):
    """Plan, rows and layer in one graph: its replays follow the requests' new tokens of their time, as calls do."""
    d, B, page, cols, n = 256, 5, 4, 12, 12
    layer, _, _ = _served(cuda_dev, d, 512, 4, 2, 64)
    x = _rand(cuda_dev, n, d, seed=81)
    labels = torch.tensor([1, -1, 0, 2, 1], dtype=I32, device=cuda_dev)
    news = torch.tensor(STEPS, dtype=I32, device=cuda_dev)

    def world():
        return (binding.PagePool.full(B * cols, page, cuda_dev), binding.KVCache.empty(B * cols, page, 2, 64, BF, cuda_dev),
                torch.full((B, cols), -1, dtype=I32, device=cuda_dev), torch.zeros(B, dtype=I32, device=cuda_dev), torch.ones(B, dtype=I32, device=cuda_dev))

    def step(pool, cache, table, lens, new, stream=None):
        p = binding.twell_kv_plan(pool, table, lens, new, n, labels=labels, stream=stream)
        rows, seen = p.per_token(table, lens, stream=stream)
        return layer.decode(x, None, cache, p.slots, rows, seen, positions=p.positions, adapter_ids=p.owner, stream=stream)

    w, want = world(), []
    for new in news:
        w[4].copy_(new)
        want.append([t.clone() for t in step(*w)])
    v, side = world(), torch.cuda.Stream()
    torch.cuda.synchronize()
    other = world()
    torch.cuda.synchronize()
    step(*other, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(*v)
    for i, new in enumerate(news):
        v[4].copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
    assert torch.equal(v[2], w[2]) and torch.equal(v[3], w[3]) and torch.equal(v[0].state, w[0].state)
