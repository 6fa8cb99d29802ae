"""The plan of a step on the GPU (twell_kv_plan): every output equals, integer for integer, what a walk over the requests one
after the other gives, including what is refused."""
import random

import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, build

pytestmark = pytest.mark.gpu
I32 = torch.int32
EMPTY, CHECK = 8, 5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()


def _walk(ring, state, page, table, lens, new, M, labels=None):
    """The definition: (slots, positions, owner, starts, table, lens, ring, state, {recorded codes})."""
    ring, table, lens = list(ring), [list(r) for r in table], list(lens)
    n, cols = len(ring), len(table[0])
    head, free = state[0], state[1]
    codes = set()
    if not (0 <= free <= n and 0 <= head and (head < n or head == free == 0)):
        head, free = 0, 0
        codes.add(CHECK)
    slots, positions, owner = [-1] * M, [0] * M, [-1] * M
    cap = min(cols * page, 2 ** 31 - 1024)
    starts, at, wanted, taken = [], 0, 0, 0
    gives = []
    for b, (past, add) in enumerate(zip(list(lens), new)):
        starts.append(min(at, 2 ** 31 - 1))
        count, begin = max(add, 0), at
        at += count
        ok = add >= -1 and 0 <= past and past + count <= cap and (count == 0 or at <= M)
        if not ok:
            codes.add(CHECK)
        held = -(-past // page)
        if ok and add == -1:
            gives.append((b, held))
        served = ok and add >= 0
        if ok and count:
            need = -(-(past + count) // page) - held
            if need and wanted + need > free:
                codes.add(EMPTY)
                served = False
            elif need:
                for p in range(need):
                    table[b][held + p] = ring[(head + wanted + p) % n]
                taken = wanted + need
            wanted += need
        for i in range(min(count, max(0, M - begin))):
            owner[begin + i] = labels[b] if labels is not None else b
            if served:
                positions[begin + i] = past + i
                pg = table[b][(past + i) // page]
                if 0 <= pg < n:
                    slots[begin + i] = pg * page + (past + i) % page
                else:
                    codes.add(CHECK)
        if served:
            lens[b] = past + count
    starts.append(min(at, 2 ** 31 - 1))
    back = sum(h for _, h in gives)
    if free + back > n:
        codes.add(CHECK)
        gives, back = [], 0
    j = head + free
    for b, held in gives:
        lens[b] = 0
        for p in range(held):
            if not 0 <= table[b][p] < n:
                codes.add(CHECK)
            ring[j % n] = table[b][p]
            j += 1
    return slots, positions, owner, starts, table, lens, ring, [(head + taken) % max(n, 1), free - taken + back, 0, 0], codes


def _run(dev, ring, state, page, table, lens, new, M, labels=None, in_place=True):
    t = lambda v: torch.tensor(v, dtype=I32).to(dev)  # noqa: E731
    pool = binding.PagePool(t(ring), t(state), page)
    table, lens_, new_ = t(table), t(lens), t(new)
    status = torch.zeros(1, dtype=I32, device=dev)
    lo, so = (None, None) if in_place else (torch.full_like(lens_, 99), torch.full_like(pool.state, 99))
    # rows that the call has to write, all of them
    plan = binding.StepPlan(*(torch.full((M,), 12345, dtype=I32, device=dev) for _ in range(3)),
                            torch.full((len(lens) + 1,), 12345, dtype=I32, device=dev))
    p = binding.twell_kv_plan(pool, table, lens_, new_, M, labels=None if labels is None else t(labels), plan=plan,
                              seq_lens_out=lo, state_out=so, status=status)
    if not in_place:
        assert lens_.tolist() == list(lens) and pool.state.tolist() == list(state)
    return (p.slots.tolist(), p.positions.tolist(), p.owner.tolist(), p.starts.tolist(), table.tolist(),
            (lens_ if in_place else lo).tolist(), pool.ring.tolist(), (pool.state if in_place else so).tolist(),
            binding.twell_read_status(status))


def _same(got, want):
    names = ("slots", "positions", "owner", "starts", "table", "lens", "ring", "state")
    for name, g, w in zip(names, got, want):
        assert g == w, name
    assert got[8] in want[8] or (got[8] == 0 and not want[8])


def _make(seed, B, page, past, new, spare=5, cols=0):
    r = random.Random(seed)
    lens = [r.randint(0, past) for _ in range(B)]
    new = [new(r) for _ in range(B)]
    held = [-(-n // page) for n in lens]
    need = [max(0, -(-(n + max(a, 0)) // page) - h) for n, a, h in zip(lens, new, held)]
    n = sum(held) + max(0, sum(need) + spare)
    pages = list(range(n))
    r.shuffle(pages)
    cols = max(cols, max(h + x for h, x in zip(held, need)), 1)
    table = [[-1] * cols for _ in range(B)]
    for b in range(B):
        table[b][:held[b]] = [pages.pop() for _ in range(held[b])]
    head = r.randrange(n) if n else 0
    ring = [-1] * n
    for i, p in enumerate(pages):
        ring[(head + i) % n] = p
    return ring, [head, len(pages), 0, 0], table, lens, new


def _mixed(r):
    u = r.random()
    return -1 if u < 0.2 else 0 if u < 0.3 else r.randint(2, 90) if u < 0.5 else 1


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("page", [1, 8, 64])
@pytest.mark.parametrize("B", [1, 2, 31, 33, 500, 513, 1500])
def test_steps(cuda_dev, B, page, in_place):
    ring, state, table, lens, new = _make(B + page, B, page, 200, _mixed)
    total = sum(max(a, 0) for a in new)
    for M in (total, total + 77):
        want = _walk(ring, state, page, table, lens, new, M)
        assert not want[8]
        _same(_run(cuda_dev, ring, state, page, table, lens, new, M, in_place=in_place), want)


def test_many_requests(cuda_dev):
    ring, state, table, lens, new = _make(3, 4096, 16, 40, _mixed)
    labels = [b % 7 - 1 for b in range(4096)]
    M = sum(max(a, 0) for a in new) + 3
    for in_place in (True, False):
        _same(_run(cuda_dev, ring, state, 16, table, lens, new, M, labels, in_place), _walk(ring, state, 16, table, lens, new, M, labels))


@pytest.mark.parametrize("page", [16, 64])
def test_long_prompts(cuda_dev, page):
    """More tokens than one block takes."""
    ring, state, table, lens, new = _make(page, 7, page, 300, lambda r: r.randint(1, 12000))
    M = sum(new) + 1
    _same(_run(cuda_dev, ring, state, page, table, lens, new, M), _walk(ring, state, page, table, lens, new, M))


def test_steps_one_after_the_other(cuda_dev):
    """A server's life: requests arrive, grow, end and their pages come round again; the ring turns several times."""
    r = random.Random(5)
    page, B, n, cols = 4, 24, 120, 12
    ring, state = list(range(n)), [0, n, 0, 0]
    table, lens = [[-1] * cols for _ in range(B)], [0] * B
    t = lambda v: torch.tensor(v, dtype=I32).to(cuda_dev)  # noqa: E731
    pool, dt, dl = binding.PagePool.full(n, page, cuda_dev), t(table), t(lens)
    status = torch.zeros(1, dtype=I32, device=cuda_dev)
    M = 200
    for _ in range(120):
        new = [-1 if x > 30 else r.choice([1, 1, 1, 0, 5]) if x else r.choice([0, 0, 9]) for x in lens]
        while sum(max(a, 0) for a in new) > M:
            new[new.index(max(new))] = 0
        p = binding.twell_kv_plan(pool, dt, dl, t(new), M, status=status)
        slots, positions, owner, starts, table, lens, ring, state, codes = _walk(ring, state, page, table, lens, new, M)
        code = binding.twell_read_status(status)
        _same((p.slots.tolist(), p.positions.tolist(), p.owner.tolist(), p.starts.tolist(), dt.tolist(), dl.tolist(),
               pool.ring.tolist(), pool.state.tolist(), code), (slots, positions, owner, starts, table, lens, ring, state, codes))
    # no page has two holders, and none is lost
    held = [table[b][i] for b in range(B) for i in range(-(-lens[b] // page))]
    free = [ring[(state[0] + i) % n] for i in range(state[1])]
    assert sorted(held + free) == list(range(n))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("spare", [-1, -3, -20, -200])
def test_too_few_pages(cuda_dev, spare, in_place):
    ring, state, table, lens, new = _make(9, 60, 8, 100, lambda r: r.choice([1, 1, 20]), spare=spare)
    M = sum(new)
    want = _walk(ring, state, 8, table, lens, new, M)
    assert want[8] == {EMPTY}
    _same(_run(cuda_dev, ring, state, 8, table, lens, new, M, in_place=in_place), want)


def test_requests_that_are_refused(cuda_dev):
    """Lengths, new tokens and ends that cannot be, one at a time and together; the others are served."""
    page = 8
    for seed, spoil in enumerate(({2: ("len", -3)}, {2: ("len", 10 ** 6)}, {2: ("new", -2)}, {2: ("new", 2 ** 31 - 1)}, {0: ("len", -1), 5: ("new", 900)},
                                  {3: ("new", -2 ** 31)}, {2: ("new", 2 ** 31 - 1), 4: ("new", 2 ** 31 - 1), 6: ("new", 2 ** 31 - 1)})):
        ring, state, table, lens, new = _make(seed, 9, page, 100, lambda r: r.choice([1, 0, 17, -1]), cols=20)
        M = sum(max(a, 0) for a in new)
        for b, (what, v) in spoil.items():
            (lens if what == "len" else new)[b] = v
        want = _walk(ring, state, page, table, lens, new, M)
        assert CHECK in want[8]
        _same(_run(cuda_dev, ring, state, page, table, lens, new, M), want)


def test_lengths_near_32_bits(cuda_dev):
    """A row of 2^21 pages of 1024 tokens: the last length that is taken, and the first that is not."""
    cols, page = 1 << 21, 1024
    table = torch.zeros((2, cols), dtype=I32, device=cuda_dev)
    table[0, cols - 2] = 5
    lens = torch.tensor([2 ** 31 - 1025, 2 ** 31 - 1024], dtype=I32, device=cuda_dev)
    status = torch.zeros(1, dtype=I32, device=cuda_dev)
    pool = binding.PagePool.full(8, page, cuda_dev)
    p = binding.twell_kv_plan(pool, table, lens, torch.ones_like(lens), 2, status=status)
    assert p.positions.tolist() == [2 ** 31 - 1025, 0] and p.slots.tolist() == [5 * 1024 + 1023, -1]
    assert lens.tolist() == [2 ** 31 - 1024] * 2 and pool.state.tolist() == [0, 8, 0, 0] and binding.twell_read_status(status) == CHECK


def test_rows_that_do_not_hold_the_step(cuda_dev):
    ring, state, table, lens, new = _make(4, 12, 8, 50, lambda r: r.randint(1, 9))
    for M in (0, 1, sum(new) - 1, sum(new[:6])):
        want = _walk(ring, state, 8, table, lens, new, M)
        assert want[8] == {CHECK}
        _same(_run(cuda_dev, ring, state, 8, table, lens, new, M), want)


def test_bad_pages_and_pools(cuda_dev):
    ring, state, table, lens, new = _make(6, 10, 8, 60, lambda r: r.choice([3, 9, -1]))
    n, M = len(ring), sum(max(a, 0) for a in new)
    # a page that does not exist, in a row and in the ring
    for bad in (n, -5, 2 ** 31 - 1):
        rows = [list(x) for x in table]
        for b in range(10):
            if lens[b]:
                rows[b][(lens[b] - 1) // 8] = bad
        _same(_run(cuda_dev, ring, state, 8, rows, lens, new, M), _walk(ring, state, 8, rows, lens, new, M))
        cells = list(ring)
        cells[state[0]] = bad
        _same(_run(cuda_dev, cells, state, 8, table, lens, new, M), _walk(cells, state, 8, table, lens, new, M))
    # pages given back that are free already; a state outside the ring
    for other in ([state[0], n, 0, 0], [n, 1, 0, 0], [-1, 2, 0, 0], [0, -1, 0, 0], [0, n + 1, 0, 0]):
        want = _walk(ring, other, 8, table, lens, new, M)
        assert CHECK in want[8]
        _same(_run(cuda_dev, ring, other, 8, table, lens, new, M), want)


def test_no_requests_and_no_pages(cuda_dev):
    _same(_run(cuda_dev, [3, 1, 0, 2], [2, 3, 0, 0], 8, [[0]], [0], [0], 5), _walk([3, 1, 0, 2], [2, 3, 0, 0], 8, [[0]], [0], [0], 5))
    pool = binding.PagePool.full(0, 16, cuda_dev)
    e = torch.empty(0, dtype=I32, device=cuda_dev)
    p = binding.twell_kv_plan(pool, torch.empty((0, 4), dtype=I32, device=cuda_dev), e, e, 6)
    assert p.slots.tolist() == [-1] * 6 and p.positions.tolist() == [0] * 6 and p.owner.tolist() == [-1] * 6 and p.starts.tolist() == [0]
    assert pool.state.tolist() == [0, 0, 0, 0]
    status = torch.zeros(1, dtype=I32, device=cuda_dev)
    lens = torch.zeros(1, dtype=I32, device=cuda_dev)
    binding.twell_kv_plan(pool, torch.zeros((1, 4), dtype=I32, device=cuda_dev), lens, lens + 1, 1, status=status)
    assert binding.twell_read_status(status) == EMPTY and lens.tolist() == [0]


def test_refusals(cuda_dev):
    pool = binding.PagePool.full(8, 16, cuda_dev)
    i = lambda *s: torch.zeros(s, dtype=I32, device=cuda_dev)  # noqa: E731
    f = binding.twell_kv_plan
    for bad in (lambda: f(pool, i(2), i(2), i(2), 4), lambda: f(pool, i(2, 3), i(3), i(2), 4), lambda: f(pool, i(2, 3), i(2).long(), i(2), 4),
                lambda: f(pool, i(2, 3), i(2), i(2).cpu(), 4), lambda: f(pool, i(2, 3), i(2), i(2), 4, labels=i(3)),
                lambda: f(pool, i(3, 2).t(), i(2), i(2), 4), lambda: f(binding.PagePool(pool.ring, i(2), 16), i(2, 3), i(2), i(2), 4),
                lambda: f(pool, i(2, 3), i(2), i(2), 4, plan=binding.StepPlan(i(4), i(3), i(4), i(3))),
                lambda: f(pool, i(2, 3), i(2), i(2), 4, seq_lens_out=i(1))):
        with pytest.raises(ValueError):
            bad()
    for bad, code in ((lambda: f(binding.PagePool(pool.ring, pool.state, 12), i(2, 3), i(2), i(2), 4), 2),
                      (lambda: f(pool, i(4097, 1), i(4097), i(4097), 4), 2), (lambda: f(pool, i(2, 0), i(2), i(2), 4), 1),
                      (lambda: (lambda n: f(pool, i(2, 3), i(2), n, 4, seq_lens_out=n))(i(2)), 1)):
        with pytest.raises(binding.TwellError) as e:
            bad()
        assert e.value.code == code
    assert pool.state.tolist() == [0, 8, 0, 0] and binding.twell_read_status() == 0
