"""GPU parity of the low-rank adapters (twell_lora_add) against the formula in 64 bits.

x, a and b enter exactly and products are exact in fp32; a sum of n terms in any order and with truncating additions stays
within n 2^-22 of the sum of its terms' sizes. t = a x enters the second product with 16 bits or more (two bf16 parts: what a
half step of 2^-8 leaves is rounded to a half step of 2^-8 again), its scale is one rounding. y is added in fp32 and the
result rounded once to bf16 (2^-8)."""
import pytest
import torch

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


def _rand(dev, *shape, seed, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(BF).to(dev)


def _adapters(dev, L, R, k, n, seed, ragged=False):
    g = torch.Generator("cpu").manual_seed(seed)
    ranks = None
    if ragged:
        ranks = torch.randint(0, R + 1, (L,), generator=g).to(I32)
        ranks[0] = R
    a, b = _rand(dev, L, R, k, seed=seed + 1, scale=k ** -0.5), _rand(dev, L, n, R, seed=seed + 2, scale=R ** -0.5)
    scale = torch.randn(L, generator=g).to(dev)
    if ragged:
        for i, r in enumerate(ranks.tolist()):  # what lies past a rank may be anything
            a[i, r:] = float("nan")
            b[i, :, r:] = float("inf")
        ranks = ranks.to(dev)
    return binding.Adapters(a, b, scale, ranks)


def _ids(dev, N, L, seed, form):
    g = torch.Generator("cpu").manual_seed(seed)
    if form == "one":
        ids = torch.full((N,), L - 1)
    elif form == "runs":
        ids = torch.randint(-1, L, (N // 37 + 1,), generator=g).repeat_interleave(37)[:N]
    else:
        ids = torch.randint(-1, L, (N,), generator=g)
    return ids.to(I32).to(dev)


def _check(got, y, x, ad, ids):
    for i in range(-1, ad.a.shape[0]):
        rows = (ids == i).nonzero()[:, 0]
        if not len(rows):
            continue
        if i < 0:
            assert torch.equal(got[rows], y[rows])
            continue
        r = ad.a.shape[1] if ad.ranks is None else int(ad.ranks[i])
        A, B, s = ad.a[i, :r].double(), ad.b[i, :, :r].double(), float(ad.scale[i])
        X, Y = x[rows].double(), y[rows].double()
        t = X @ A.t()
        off = X.shape[1] * 2.0 ** -22 * (X.abs() @ A.abs().t()) + (2.0 ** -16 + 2.0 ** -23) * t.abs()
        ref = Y + s * (t @ B.t())
        room = abs(s) * (off @ B.abs().t() + max(r, 1) * 2.0 ** -22 * (t.abs() @ B.abs().t())) + 2.0 ** -23 * (Y.abs() + ref.abs())
        bound = room + 2.0 ** -8 * (ref.abs() + room)
        err = (got[rows].double() - ref).abs()
        assert (err <= bound).all(), (i, (err / bound).max().item())


# widths about the tiles' ends, ranks of one to eight 16-row pieces
@pytest.mark.parametrize("form", ["any", "one"])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("k,n,R", [(8, 8, 8), (64, 40, 16), (200, 264, 24), (512, 2048, 32), (2048, 512, 64), (1000, 136, 128), (24, 1000, 40)])
@pytest.mark.parametrize("N", [1, 2, 9, 16, 17, 40])
def test_decode_batches(cuda_dev, N, k, n, R, ragged, form):
    L = 6
    ad = _adapters(cuda_dev, L, R, k, n, seed=k + R, ragged=ragged)
    ids = _ids(cuda_dev, N, L, N + k, form)
    x, y = _rand(cuda_dev, N, k, seed=N), _rand(cuda_dev, N, n, seed=N + 1)
    out = torch.full_like(y, 7.0)
    assert binding.twell_lora_add(y, x, ad, ids, out=out) is out
    _check(out, y, x, ad, ids)
    z = y.clone()
    assert binding.twell_lora_add(z, x, ad, ids) is z and torch.equal(z, out)


@pytest.mark.parametrize("form", ["any", "one", "runs"])
@pytest.mark.parametrize("N,k,n,R,L", [(65, 128, 64, 16, 3), (257, 520, 264, 8, 40), (513, 256, 136, 24, 2), (700, 264, 512, 128, 5), (1025, 72, 80, 64, 300),
                                       (513, 136, 264, 16, 16), (700, 264, 136, 32, 22), (991, 520, 1032, 64, 4000), (1024, 2048, 72, 128, 64),
                                       (2000, 512, 520, 32, 4), (5000, 136, 264, 16, 9)])
def test_larger_batches(cuda_dev, N, k, n, R, L, form):
    for ragged in (False, True):
        ad = _adapters(cuda_dev, L, R, k, n, seed=N, ragged=ragged)
        ids = _ids(cuda_dev, N, L, N + 1, form)
        x, y = _rand(cuda_dev, N, k, seed=N + 2), _rand(cuda_dev, N, n, seed=N + 3)
        out = binding.twell_lora_add(y, x, ad, ids, out=torch.full_like(y, 7.0))
        _check(out, y, x, ad, ids)
        assert torch.equal(binding.twell_lora_add(y.clone(), x, ad, ids), out)


@pytest.mark.parametrize("N,L,R", [(30, 4096, 16), (400, 4096, 64), (3000, 4096, 8), (512, 1, 128), (16384, 3, 16), (16384 + 777, 40, 24),
                                   (33000, 2, 128)])
def test_many_adapters_and_many_tokens(cuda_dev, N, L, R):
    """Up to 4096 adapters, and batches of several passes."""
    k, n = 64, 72
    ad = _adapters(cuda_dev, L, R, k, n, seed=N, ragged=True)
    ids = _ids(cuda_dev, N, L, N + 1, "any")
    x, y = _rand(cuda_dev, N, k, seed=N + 2), _rand(cuda_dev, N, n, seed=N + 3)
    out = binding.twell_lora_add(y, x, ad, ids, out=torch.full_like(y, 7.0))
    # the formula for all tokens at once: t of a token's own adapter, what lies past its rank left out
    own = ids.long().clamp_min(0)
    low = torch.arange(R, device=cuda_dev) < ad.ranks[own][:, None]
    use = low & (ids >= 0)[:, None]
    for rows in torch.arange(N, device=cuda_dev).split(4096):
        i, u, X, Y = own[rows], use[rows], x[rows].double(), y[rows].double()
        A, B = ad.a[i].double().masked_fill(~u[..., None], 0), ad.b[i].double().masked_fill(~u[:, None], 0)
        s = ad.scale[i].double()[:, None]
        t = torch.einsum("mrk,mk->mr", A, X)
        off = k * 2.0 ** -22 * torch.einsum("mrk,mk->mr", A.abs(), X.abs()) + (2.0 ** -16 + 2.0 ** -23) * t.abs()
        ref = Y + s * torch.einsum("mnr,mr->mn", B, t)
        room = s.abs() * (torch.einsum("mnr,mr->mn", B.abs(), off + R * 2.0 ** -22 * t.abs())) + 2.0 ** -23 * (Y.abs() + ref.abs())
        err = (out[rows].double() - ref).abs()
        assert (err <= room + 2.0 ** -8 * (ref.abs() + room)).all()
    assert torch.equal(out[ids < 0], y[ids < 0])
    assert torch.equal(binding.twell_lora_add(y.clone(), x, ad, ids), out)


@pytest.mark.parametrize("N", [1, 12, 100, 300, 1500])
def test_a_row_does_not_depend_on_the_others(cuda_dev, N):
    """The same bits in another order, beside other rows, and whatever the others hold."""
    k, n, R, L = 640, 328, 32, 5
    ad = _adapters(cuda_dev, L, R, k, n, seed=1)
    ids = _ids(cuda_dev, N, L, 2, "any")
    x, y = _rand(cuda_dev, N, k, seed=3), _rand(cuda_dev, N, n, seed=4)
    out = binding.twell_lora_add(y, x, ad, ids, out=torch.empty_like(y))
    assert torch.equal(binding.twell_lora_add(y, x, ad, ids, out=torch.empty_like(y)), out)
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(5)).to(cuda_dev)
    assert torch.equal(binding.twell_lora_add(y[perm], x[perm], ad, ids[perm], out=torch.empty_like(y)), out[perm])
    if N > 1:
        x[1], y[N // 2 + 1 if N > 2 else 0, 3] = float("nan"), float("inf")
        spoilt = binding.twell_lora_add(y, x, ad, ids, out=torch.empty_like(y))
        keep = torch.ones(N, dtype=torch.bool, device=cuda_dev)
        keep[1] = keep[N // 2 + 1 if N > 2 else 0] = False
        assert torch.equal(spoilt[keep], out[keep])
        assert int(ids[1]) < 0 or torch.isnan(spoilt[1]).all()


@pytest.mark.parametrize("N,R", [(3, 16), (16, 64), (300, 64), (1000, 16), (1000, 128), (1500, 32)])
def test_replays_take_the_ids_of_their_time(cuda_dev, N, R):
    """A captured call, replayed with other ids: few adapters and many, long runs, none at all. The blocks share what tiles there are."""
    k, n, L = 648, 1032, 40
    ad = _adapters(cuda_dev, L, R, k, n, seed=R, ragged=True)
    x, y = _rand(cuda_dev, N, k, seed=1), _rand(cuda_dev, N, n, seed=2)
    out, ids = torch.empty_like(y), _ids(cuda_dev, N, L, 3, "any")
    binding.twell_lora_add(y, x, ad, ids, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.twell_lora_add(y, x, ad, ids, out=out)
    kinds = [_ids(cuda_dev, N, L, 4, "runs"), torch.full_like(ids, -1), _ids(cuda_dev, N, L, 5, "one"), _ids(cuda_dev, N, L, 6, "any")]
    got = []
    for other in kinds * 3:  # without a wait between them
        ids.copy_(other)
        graph.replay()
        got.append(out.clone())
    for other, o in zip(kinds * 3, got):
        assert torch.equal(o, binding.twell_lora_add(y, x, ad, other, out=torch.empty_like(y)))
    _check(got[0], y, x, ad, kinds[0])
    _check(got[3], y, x, ad, kinds[3])
    assert torch.equal(got[1], y)


@pytest.mark.parametrize("N", [5, 80, 900])
def test_slices_of_wider_rows(cuda_dev, N):
    """Rows of a fused projection: the columns beside the slice stay, and rows without an adapter are not written."""
    k, n, L = 256, 264, 3
    ad = _adapters(cuda_dev, L, 16, k, n, seed=7)
    ids = _ids(cuda_dev, N, L, 8, "any")
    xw, yw = _rand(cuda_dev, N, 2 * k, seed=9), _rand(cuda_dev, N, 3 * n, seed=10)
    x, y = xw[:, k:], yw[:, n:2 * n]
    want = binding.twell_lora_add(y.contiguous(), x.contiguous(), ad, ids)
    keep = yw.clone()
    binding.twell_lora_add(y, x, ad, ids)
    assert torch.equal(y, want)
    assert torch.equal(yw[:, :n], keep[:, :n]) and torch.equal(yw[:, 2 * n:], keep[:, 2 * n:])
    _check(y, keep[:, n:2 * n], x, ad, ids)


@pytest.mark.parametrize("N", [3, 70, 600])
def test_what_is_not_finite(cuda_dev, N):
    """An infinite t goes on as one: inf - inf of its parts must not make a NaN of it."""
    k, n = 64, 48
    a, b = torch.zeros((2, 8, k), dtype=BF, device=cuda_dev), torch.zeros((2, n, 8), dtype=BF, device=cuda_dev)
    a[:, 0, 0], b[:, :, 0] = 1.0, 2.0
    ad = binding.Adapters(a, b, torch.ones(2, device=cuda_dev))
    x, y = torch.zeros((N, k), dtype=BF, device=cuda_dev), torch.zeros((N, n), dtype=BF, device=cuda_dev)
    x[0, 0], x[1, 0], x[2, 0] = float("inf"), float("nan"), 3.0
    ids = torch.tensor([0, 0, 1] + [0] * (N - 3), dtype=I32, device=cuda_dev)
    out = binding.twell_lora_add(y, x, ad, ids)
    # 0 x inf in the other products of a row is NaN where the formula has it so: t = a x has a[0, 0] = 1 and zeros elsewhere
    assert torch.isnan(out[1]).all() and (out[2] == 6.0).all() and (out[3:] == 0).all()
    a[:, 1:] = 1.0  # every t of an infinite x is infinite, and b's other columns must not be zero for the sum to be
    b[:] = 1.0
    x[0] = 0
    x[0, 0] = float("inf")
    a[:, :, 1:] = 1.0
    out = binding.twell_lora_add(torch.zeros_like(y), x, ad, ids)
    assert (out[0] == float("inf")).all()


def test_ids_and_ranks_that_do_not_exist(cuda_dev):
    k, n, L = 64, 72, 3
    for N in (6, 100, 800):
        ad = _adapters(cuda_dev, L, 16, k, n, seed=11)
        x, y = _rand(cuda_dev, N, k, seed=12), _rand(cuda_dev, N, n, seed=13)
        ids = _ids(cuda_dev, N, L, 14, "any")
        for bad in (L, -2, 2 ** 31 - 1, -2 ** 31):
            other = ids.clone()
            other[N - 2] = bad
            as_none = ids.clone()
            as_none[N - 2] = -1
            status = torch.zeros(1, dtype=I32, device=cuda_dev)
            out = binding.twell_lora_add(y, x, ad, other, out=torch.empty_like(y), status=status)
            assert binding.twell_read_status(status) == 5
            assert torch.equal(out, binding.twell_lora_add(y, x, ad, as_none, out=torch.empty_like(y)))
        for bad in (17, -1):
            ranks = torch.tensor([16, bad, 16], dtype=I32, device=cuda_dev)
            status = torch.zeros(1, dtype=I32, device=cuda_dev)
            ids[0] = 1
            out = binding.twell_lora_add(y, x, binding.Adapters(ad.a, ad.b, ad.scale, ranks), ids, out=torch.empty_like(y), status=status)
            assert binding.twell_read_status(status) == 5
            none = torch.where(ids == 1, -1, ids)
            assert torch.equal(out, binding.twell_lora_add(y, x, ad, none, out=torch.empty_like(y)))


def test_refusals(cuda_dev):
    ad = _adapters(cuda_dev, 2, 16, 64, 32, seed=15)
    x, y, ids = (torch.zeros((4, c), dtype=BF, device=cuda_dev) for c in (64, 32, 1))
    ids = torch.zeros(4, dtype=I32, device=cuda_dev)
    f = binding.twell_lora_add
    for bad in (lambda: f(y, x[:, :56], ad, ids), lambda: f(y[:, :24], x, ad, ids), lambda: f(y.float(), x, ad, ids), lambda: f(y, x.half(), ad, ids),
                lambda: f(y, x, ad, ids.long()), lambda: f(y, x, ad, ids[:3]), lambda: f(y, x, ad, ids.cpu()), lambda: f(y[:3], x, ad, ids),
                lambda: f(y, x[0], ad, ids), lambda: f(y, x, ad, ids, out=y[:, :24]), lambda: f(y, x.t().contiguous().t(), ad, ids),
                lambda: f(y, x, binding.Adapters(ad.a, ad.b[:, :, :8], ad.scale), ids), lambda: f(y, x, binding.Adapters(ad.a, ad.b, ad.scale[:1]), ids),
                lambda: f(y, x, binding.Adapters(ad.a, ad.b, ad.scale, ids), ids)):
        with pytest.raises(ValueError):
            bad()
    assert f(y[:0], x[:0], ad, ids[:0]).shape == (0, 32)
    wide = torch.zeros((4, 100), dtype=BF, device=cuda_dev)
    for bad in (lambda: f(wide[:, 4:36], x, ad, ids), lambda: f(wide[:, :32], x, ad, ids)):
        with pytest.raises(binding.TwellError) as e:
            bad()
        assert e.value.code == 1
