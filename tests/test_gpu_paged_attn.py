"""GPU parity of the one-token attention over the paged cache (twell_paged_attn_decode) against the formula in
64 bits.

Bounds. A score is an fp32 sum of hd exact products: e = scale hd 2^-22 max_t sum|q k| (any order, truncating
additions), plus 2^-20 for its scaling, the maximum's subtraction and the exponential (|score| <= 2^7 here, so a few
2^-24 |score| are below 2^-15: the constant is 2^-14). A weight is so off by 2e + 2^-14 relative; its rounding adds
2^-16 with a bf16 cache (hi + lo parts) and 2^-11 with an e4m3 one (fp16), plus 2^-25 of the largest weight for
those under fp16's normal range; the query's rounding to fp16 under a common power of two adds 2^-25 max|q| per
element: hd 2^-24 max|q| max|k| scale. out is then within twice the weights' error times sum p |v|, sums included, plus
one bf16 rounding, 2^-8 |out|. lse is within e + 2^-14.
The bounds of an e4m3 cache are those of one fp16 part under a largest weight of 1; with two parts under 2^15, as they are,
the tests of many small weights and of values of very different sizes hold it to more.
"""
import math

import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()
    binding.status_buffer(cuda_dev).zero_()
    yield
    assert binding.twell_read_status() == 0, "device status was raised"


class Case:
    """A cache whose pages are handed out at random; slots that no sequence sees hold NaN (codes and scales),
    table entries past a sequence's pages hold nonsense."""

    def __init__(self, dev, lens, H, G, hd, ps, dtype, seed=0, k_size=1.0, layout="heads", v_spread=0.0, extra_cols=2):
        g = torch.Generator("cpu").manual_seed(seed)
        self.lens, self.H, self.G, self.hd, self.ps = lens, H, G, hd, ps
        B = len(lens)
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g)
        cols = max(max(need), 1) + extra_cols
        table = torch.full((B, cols), -12345678, dtype=torch.int32)
        at = 0
        self.k64, self.v64 = [], []
        shape = (pages, ps, H, hd) if layout == "tokens" else (pages, H, ps, hd)
        perm_of = (0, 2, 1, 3) if layout == "tokens" else (0, 1, 2, 3)
        host = [torch.full(shape, float("nan")).permute(perm_of) for _ in range(2)]
        scales = [torch.full((pages, H, ps), float("nan")) for _ in range(2)]
        for b, n in enumerate(lens):
            table[b, :need[b]] = perm[at:at + need[b]].to(torch.int32)
            pos = torch.arange(n)
            pg, off = table[b, pos // ps].long(), pos % ps
            for i, size in ((0, k_size), (1, 1.0)):
                x = size * torch.randn((n, H, hd), generator=g)
                if v_spread and i == 1:
                    x *= torch.exp(v_spread * torch.randn((n, H, 1), generator=g))
                if dtype == BF:
                    x = x.to(BF)
                    host[i][pg, :, off] = x.float()
                    x = x.double()
                else:
                    s = x.abs().amax(-1).clamp_min(2.0 ** -60) / 448
                    q = (x / s[..., None]).to(E4)
                    host[i][pg, :, off] = q.float()
                    scales[i][pg, :, off] = s
                    x = q.double() * s.double()[..., None]
                (self.k64, self.v64)[i].append(x)
            at += need[b]
        # the layout as asked for, kept by the copy to the device
        k, v = (torch.empty_strided(t.shape, t.stride(), dtype=dtype, device=dev) for t in host)
        for t, h in ((k, host[0]), (v, host[1])):
            t.copy_(h.to(dtype))
        self.cache = binding.KVCache(k, v) if dtype == BF else binding.KVCache(k, v, *(s.to(dev) for s in scales))
        self.table = table.to(dev)
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.q = torch.randn((B, H * G, hd), generator=g).to(BF).to(dev)
        self.dtype = dtype

    def run(self, **kw):
        lse = torch.full(self.q.shape[:2], 7.0, dtype=F32, device=self.q.device)
        out, lse = binding.twell_paged_attn_decode(self.q, self.cache, self.table, self.lens_d, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, window=0, scale=None, q=None):
        scale = scale if scale is not None else 1 / math.sqrt(self.hd)
        q64 = (q if q is not None else self.q).cpu().double()
        out, lse = out.cpu().double(), lse.cpu().double()
        for b, n in enumerate(self.lens):
            lo = max(0, n - window) if window else 0
            o = out[b].view(self.H, self.G, self.hd)
            le = lse[b].view(self.H, self.G)
            if n == 0:
                assert torch.count_nonzero(o) == 0 and (le == -math.inf).all()
                continue
            k, v = self.k64[b][lo:], self.v64[b][lo:]
            qb = q64[b].view(self.H, self.G, self.hd)
            z = scale * torch.einsum("hgd,nhd->hgn", qb, k)
            rl = torch.logsumexp(z, -1)
            p = torch.exp(z - rl[..., None])
            ro = torch.einsum("hgn,nhd->hgd", p, v)
            mass = torch.einsum("hgn,nhd->hgd", p, v.abs())
            e = scale * self.hd * 2.0 ** -22 * torch.einsum("hgd,nhd->hgn", qb.abs(), k.abs()).amax(-1)
            w = 2 * e + 2.0 ** -14
            if self.dtype == E4:
                e = e + scale * self.hd * 2.0 ** -24 * qb.abs().amax(-1) * k.abs().amax((0, 2))[:, None]
                w = 2 * e + 2.0 ** -14 + 2.0 ** -11
                # weights under fp16's normal range: 2^-25 of the largest weight, which stands for a mass of
                # p v = at most amax
                mass = mass + (n - lo) * 2.0 ** -14 * 2 * (p[..., None] * v.abs().amax(-1).permute(1, 0)[:, None, :, None]).amax(2)
            else:
                w = w + 2.0 ** -16
            bound = 2 * w[..., None] * mass + 2.0 ** -8 * ro.abs() + 1e-30
            err = (o - ro).abs()
            assert (err <= bound).all(), (b, n, (err / bound).max().item(), err.max().item())
            assert ((le - rl).abs() <= e + 2.0 ** -14).all(), (b, n, (le - rl).abs().max().item())


LENS = [0, 1, 15, 16, 17, 33, 64, 100, 255, 257]


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("hd", [64, 96, 128, 256])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (3, 5), (1, 8), (2, 9), (1, 16), (1, 20), (5, 1), (1, 33)])
def test_head_layouts(cuda_dev, H, G, hd, dtype):
    c = Case(cuda_dev, LENS, H, G, hd, 16, dtype, seed=hd + G)
    out, lse = c.run()
    c.check(out, lse)
    again, _ = binding.twell_paged_attn_decode(c.q, c.cache, c.table, c.lens_d)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("ps", [1, 2, 8, 32, 64, 1024])
def test_page_sizes(cuda_dev, ps, dtype):
    c = Case(cuda_dev, [3, 0, 70, 129, 2048, 31], 2, 4, 128, ps, dtype, seed=ps)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("window", [1, 5, 16, 40, 100, 5000])
def test_windows(cuda_dev, window, dtype):
    """Tokens before the window do not count, and their pages are not read: the table says nonsense there."""
    c = Case(cuda_dev, [0, 1, 4, 5, 6, 16, 47, 300, 1000], 2, 3, 64, 8, dtype, seed=window)
    for b, n in enumerate(c.lens):
        c.table[b, :max(0, n - window) // 8] = 2 ** 30
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("lens", [[4000], [20000], [1], [9000, 1, 0, 3], [1600] * 7, [100 + 37 * i for i in range(40)],
                                  [5] * 300, [0] * 9])
def test_lengths_and_splits(cuda_dev, lens, dtype):
    """Long sequences over many blocks, many short ones in one warp's range, and mixtures."""
    c = Case(cuda_dev, lens, 2, 4, 128, 64, dtype, seed=len(lens))
    out, lse = c.run()
    c.check(out, lse)
    assert torch.equal(out, c.run()[0])


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("G,hd", [(16, 128), (12, 64), (8, 256), (16, 96)])
def test_long_with_many_heads(cuda_dev, G, hd, dtype):
    c = Case(cuda_dev, [7000, 12, 3000], 1, G, hd, 32, dtype, seed=G)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", [BF, E4])
def test_token_major_pages(cuda_dev, dtype):
    c = Case(cuda_dev, LENS, 4, 2, 128, 16, dtype, seed=5, layout="tokens")
    assert c.cache.k.stride(1) == 128
    c.check(*c.run())


@pytest.mark.parametrize("dtype", [BF, E4])
def test_sharp_scores_and_uneven_values(cuda_dev, dtype):
    """Scores far apart (the running maximum moves often), and values of very different sizes."""
    c = Case(cuda_dev, [1000, 333, 17], 2, 4, 64, 16, dtype, seed=8, k_size=8.0, v_spread=3.0)
    c.check(*c.run())
    c.check(*c.run(scale=0.5), scale=0.5)


def test_values_of_zeros_in_an_8bit_cache(cuda_dev):
    """Scales of zero (values that are all zeros) count in the softmax's sum and add nothing to the output."""
    c = Case(cuda_dev, [50, 20], 1, 2, 64, 16, E4, seed=9)
    for b, n in enumerate(c.lens):
        for t in range(0, n, 2 if b == 0 else 1):
            pg = int(c.table[b, t // 16])
            c.cache.v_scale[pg, 0, t % 16] = 0.0
            c.v64[b][t] = 0.0
    out, lse = c.run()
    c.check(out, lse)
    assert torch.count_nonzero(out[1]) == 0


@pytest.mark.parametrize("dtype", [BF, E4])
def test_queries_of_any_size(cuda_dev, dtype):
    """Queries beyond fp16's range, tiny ones and zeros."""
    c = Case(cuda_dev, [40, 40, 40, 40], 2, 2, 64, 16, dtype, seed=10)
    size = torch.tensor([1e9, 1e-20, 0.0, 3e-3], device=cuda_dev)[:, None, None]
    c.q = (c.q.float() * size).to(BF)
    for b, scale in ((0, 1e-10), (1, 1e18), (2, 1.0), (3, 1.0)):
        out, lse = c.run(scale=scale)
        d = Case.__new__(Case)
        d.__dict__.update(c.__dict__)
        d.lens, d.k64, d.v64 = [c.lens[b]], [c.k64[b]], [c.v64[b]]
        d.check(out[b:b + 1], lse[b:b + 1], scale=scale, q=c.q[b:b + 1])


def test_strided_queries(cuda_dev):
    """Queries as a slice of the fused projection's rows."""
    c = Case(cuda_dev, [90, 3, 20], 2, 4, 128, 16, BF, seed=11)
    row = torch.zeros((3, 12, 128), dtype=BF, device=cuda_dev)
    row[:, :8] = c.q
    out, _ = binding.twell_paged_attn_decode(row[:, :8], c.cache, c.table, c.lens_d)
    assert torch.equal(out, c.run()[0])


def test_a_key_that_is_not_finite_stays_in_its_sequence(cuda_dev):
    c = Case(cuda_dev, [60, 60, 60], 2, 4, 64, 16, BF, seed=12)
    out, lse = c.run()
    c.cache.k[int(c.table[1, 0]), 0, 5, 3] = float("nan")
    bad, bl = c.run()
    assert torch.equal(bad[[0, 2]], out[[0, 2]]) and torch.equal(bad[1, 4:], out[1, 4:])
    assert torch.isnan(bad[1, :4]).all() and torch.isnan(bl[1, :4]).all()


def test_bad_pages_and_lengths_are_reported(cuda_dev):
    c = Case(cuda_dev, [48, 48], 1, 2, 64, 16, BF, seed=13, extra_cols=0)
    good, _ = c.run()
    c.table[0, 1] = c.cache.n_pages  # its 16 tokens do not count
    out, lse = c.run()
    assert binding.twell_read_status() == 5
    assert torch.equal(out[1], good[1])
    keep = torch.cat([torch.arange(16), torch.arange(32, 48)])
    d = Case.__new__(Case)
    d.__dict__.update(c.__dict__)
    d.lens, d.k64, d.v64 = [32, 48], [c.k64[0][keep], c.k64[1]], [c.v64[0][keep], c.v64[1]]
    d.check(out, lse)
    c = Case(cuda_dev, [48, 48, 48], 1, 2, 64, 16, BF, seed=14, extra_cols=0)
    good, _ = c.run()
    c.lens_d[0], c.lens_d[2] = 49, -3  # past the table: clamped; negative: nothing
    out, lse = c.run()
    assert binding.twell_read_status() == 5
    assert torch.equal(out[:2], good[:2])
    assert torch.count_nonzero(out[2]) == 0 and (lse[2] == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF, E4])
def test_pages_past_32_bit_offsets(cuda_dev, dtype):
    """A sequence in the last pages of a cache of 2^32 + elements a kind."""
    ps, H, hd = 64, 4, 128
    pages = (1 << 32) // (ps * H * hd) + 3
    c = Case(cuda_dev, [150], H, 4, hd, ps, dtype, seed=15, extra_cols=0)
    small = c.cache
    big = [torch.empty((pages, H, ps, hd), dtype=dtype, device=cuda_dev) for _ in range(2)]
    big_s = [torch.empty((pages, H, ps), dtype=F32, device=cuda_dev) for _ in range(2)] if dtype == E4 else []
    move = torch.arange(small.n_pages, device=cuda_dev) + (pages - small.n_pages)
    for b, s in zip(big, (small.k, small.v)):
        b[pages - small.n_pages:].copy_(s)
    for b, s in zip(big_s, (small.k_scale, small.v_scale)):
        b[pages - small.n_pages:].copy_(s)
    out, _ = c.run()
    c.cache = binding.KVCache(*big, *big_s)
    c.table = move[c.table.long()].to(torch.int32)
    moved, lse = c.run()
    assert torch.equal(out, moved)
    c.check(moved, lse)


def test_side_stream(cuda_dev):
    c = Case(cuda_dev, [5000, 100, 0, 7], 4, 4, 128, 64, BF, seed=16)
    out, _ = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lse = torch.empty(c.q.shape[:2], dtype=F32, device=cuda_dev)
    other = torch.empty_like(out)
    torch.cuda.synchronize()
    binding.twell_paged_attn_decode(c.q, c.cache, c.table, c.lens_d, out=other, lse=lse, stream=s)
    s.synchronize()
    assert torch.equal(out, other)


def test_refusals(cuda_dev):
    c = Case(cuda_dev, [20, 20], 2, 2, 64, 16, BF, seed=17)
    f = binding.twell_paged_attn_decode
    for bad in (lambda: f(c.q.float(), c.cache, c.table, c.lens_d), lambda: f(c.q[:, :, :32], c.cache, c.table, c.lens_d),
                lambda: f(c.q, c.cache, c.table.long(), c.lens_d), lambda: f(c.q, c.cache, c.table[:1], c.lens_d),
                lambda: f(c.q, c.cache, c.table, c.lens_d[:1]), lambda: f(c.q, c.cache, c.table, c.lens_d, out=c.q[:1]),
                lambda: f(c.q, c.cache, c.table, c.lens_d, lse=c.q)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.TwellError) as e:
        f(c.q[:, :3].contiguous(), c.cache, c.table, c.lens_d)  # 3 query heads over 2 key heads
    assert e.value.code == 1
    with pytest.raises(binding.TwellError) as e:
        f(c.q, c.cache, c.table, c.lens_d, window=-1)
    assert e.value.code == 1
    odd = binding.KVCache(*(torch.zeros((2, 2, 16, 80), dtype=BF, device=cuda_dev) for _ in range(2)))
    with pytest.raises(binding.TwellError) as e:
        f(torch.zeros((2, 4, 80), dtype=BF, device=cuda_dev), odd, c.table, c.lens_d)  # head_dim 80
    assert e.value.code == binding.TWELL_ERR_UNSUPPORTED
    with pytest.raises(binding.TwellError) as e:
        f(c.q, c.cache, c.table, c.lens_d, ws=torch.empty(64, dtype=torch.uint8, device=cuda_dev))
    assert e.value.code == 7
    out, _ = f(c.q[:0], c.cache, c.table[:0], c.lens_d[:0])
    assert out.shape == (0, 4, 64)


def _short_lens(B, top, seed):
    """Lengths 0 .. top, with runs of empty sequences at the start, inside and at the end."""
    g = torch.Generator("cpu").manual_seed(seed)
    lens = torch.randint(0, top + 1, (B,), generator=g).tolist()
    lens[:3] = [0, 0, top]
    lens[B // 2:B // 2 + 20] = [0] * 20
    lens[-2:] = [1, 0]
    return lens


# Batches whose (sequence, key head)s are more than the SMs and few tiles each.
@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("B,H,G,hd,ps,top", [(170, 8, 3, 64, 16, 33), (100, 3, 16, 128, 32, 256), (64, 5, 7, 96, 8, 100),
                                            (90, 4, 10, 256, 32, 31), (300, 1, 1, 128, 1, 5), (400, 16, 2, 64, 32, 64)])
def test_many_short_sequences(cuda_dev, B, H, G, hd, ps, top, dtype):
    c = Case(cuda_dev, _short_lens(B, top, B), H, G, hd, ps, dtype, seed=B, extra_cols=0)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.equal(out, c.run()[0])


@pytest.mark.parametrize("dtype", [BF, E4])
def test_many_sequences_under_a_window(cuda_dev, dtype):
    c = Case(cuda_dev, _short_lens(120, 400, 3), 4, 4, 64, 16, dtype, seed=3)
    for window in (1, 31, 40, 100):
        c.check(*c.run(window=window), window=window)


def test_many_empty_sequences(cuda_dev):
    c = Case(cuda_dev, [0] * 500, 4, 4, 64, 16, BF, seed=4)
    c.check(*c.run())


def test_many_short_sequences_with_bad_lengths(cuda_dev):
    lens = _short_lens(200, 48, 6)
    c = Case(cuda_dev, lens, 2, 4, 64, 16, BF, seed=6, extra_cols=0)
    good, _ = c.run()
    full = [b for b, n in enumerate(lens) if n == 48]
    c.lens_d[full[0]], c.lens_d[199] = 1000, -7  # past the table: clamped; negative: nothing
    out, lse = c.run()
    assert binding.twell_read_status() == 5
    assert torch.equal(out, good) and (lse[199] == -math.inf).all()


def _direct(dev, k, v, q, scale):
    """One sequence over an e4m3 cache of one key head whose values are exact codes: k, v [n, hd] as power-of-two scales
    times codes; returns out, lse, the references of lse and out in 64 bits, sum p |v| and the largest p amax|v|."""
    n, hd = k.shape
    ps = 64
    pages = -(-n // ps)
    parts = []
    for x in (k, v):
        top = x.double().abs().amax(-1)
        s = torch.where(top > 0, 2.0 ** (torch.log2(top.clamp_min(1e-300)).floor() - 7), torch.ones_like(top)).float()
        codes = torch.zeros((pages * ps, hd))
        codes[:n] = x / s[:, None]
        assert torch.equal(codes[:n].to(E4).double() * s.double()[:, None], x.double())
        scales = torch.zeros(pages * ps)
        scales[:n] = s
        parts += [codes.to(E4).view(pages, 1, ps, hd).to(dev), scales.view(pages, 1, ps).to(dev)]
    cache = binding.KVCache(parts[0], parts[2], parts[1], parts[3])
    table = torch.arange(pages, dtype=torch.int32, device=dev).view(1, pages)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    lse = torch.empty((1, 1), dtype=F32, device=dev)
    out, _ = binding.twell_paged_attn_decode(q.to(BF).view(1, 1, hd).to(dev), cache, table, lens, scale=scale, lse=lse)
    z = scale * (k.double() @ q.to(BF).double())
    rl = torch.logsumexp(z, 0)
    p = torch.exp(z - rl)
    return (out.cpu().double().view(hd), lse.item(), rl.item(), p @ v.double(), p @ v.double().abs(),
            (p * v.double().abs().amax(-1)).max().item())


@pytest.mark.parametrize("n", [600, 131072])
def test_many_small_weights_in_an_8bit_cache(cuda_dev, n):
    """One token of nearly all the mass and a long tail of 2^-26 of it each, seen alone in half of the dimensions. A weight
    is off by 2^-22 of itself, 2^-40 of the largest and the score's error, here below 2^-14 as in the file's bounds: the
    tail's share is within 2^-12 of itself, and its bf16 rounding."""
    hd = 64
    k, v = torch.zeros((n, hd)), torch.zeros((n, hd))
    k[0] = 2.25 / hd  # q . k of the first token: 18, under a scale that makes it 26 in base 2
    v[0, :hd // 2] = 1.0
    v[1:, hd // 2:] = 1.0
    out, lse, rl, ro, _, _ = _direct(cuda_dev, k, v, torch.full((hd,), 8.0), 26 * math.log(2) / 18)
    assert ((out - ro).abs() <= (2.0 ** -8 + 2.0 ** -12) * ro.abs()).all(), (out, ro)
    assert abs(lse - rl) <= 2.0 ** -14


@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 26, 2.0 ** -26])
def test_values_of_very_different_sizes_in_an_8bit_cache(cuda_dev, ratio):
    """Every 50th value is `ratio` times the others, in the first half of the dimensions; the second half holds the other
    values alone. The weights' bounds of the test above; 2^-40 of the largest weight is, in values, n 2^-40 of the
    largest p amax|v|."""
    hd, n = 128, 1000
    g = torch.Generator("cpu").manual_seed(30)
    k = torch.randint(-8, 9, (n, hd), generator=g).float() / 8
    v = torch.randint(1, 16, (n, hd), generator=g).float() / 8
    v[:, 0] = v[:, hd // 2] = 15 / 8
    loud = torch.arange(n) % 50 == 7
    v[loud] *= ratio
    v[loud, hd // 2:] = 0
    v[~loud, :hd // 2] = 0
    q = torch.randint(-8, 9, (hd,), generator=g).float() / 8
    out, lse, rl, ro, mass, top = _direct(cuda_dev, k, v, q, 1 / math.sqrt(hd))
    e = hd * 2.0 ** -22 / math.sqrt(hd) * hd
    w = 2 * (2 * e + 2.0 ** -14 + 2.0 ** -20)
    err, bound = (out - ro).abs(), 2.0 ** -8 * ro.abs() + w * mass + n * 2.0 ** -40 * top
    assert (err <= bound).all(), (err / bound).max().item()
    assert abs(lse - rl) <= e + 2.0 ** -14


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_lse_does_not_depend_on_values(cuda_dev, bad, dtype):
    """A value that is not finite makes its head's output so, and leaves lse alone; sequences of the three sizes that
    a batch's forms take, the value in a full tile and in the last one."""
    lens = [9000, 70, 33]
    c = Case(cuda_dev, lens, 2, 4, 64, 16, dtype, seed=31)
    out, lse = c.run()
    for b, t in ((0, 4001), (1, 69)):
        slot = torch.tensor([int(c.table[b, t // 16]) * 16 + t % 16], dtype=torch.int32, device=cuda_dev)
        k, v = binding.twell_kv_gather(c.cache, slot)
        v[0, 1, 5] = bad
        rest = [x.view(torch.uint8) if x.dtype == E4 else x for x in
                (c.cache.k, c.cache.v[:, :1]) + (() if dtype == BF else (c.cache.k_scale, c.cache.v_scale[:, :1]))]
        kept = [x.clone() for x in rest]
        binding.twell_kv_append(c.cache, k, v, slot)
        for x, y in zip(rest, kept):  # the keys and the other head's values as they were, not rounded once more
            x.copy_(y)
    new, nl = c.run()
    # an e4m3 row with an infinity has an infinite scale: log2 of the others' stays in the running maximum, so that
    # the same sums are formed under other maxima
    assert torch.isfinite(nl).all() and ((nl - lse).abs() <= 2.0 ** -14).all()
    assert not torch.isfinite(new[:2, 4:, 5]).any()
    assert torch.equal(new[2], out[2]) and torch.equal(new[:, :4], out[:, :4])


@pytest.mark.parametrize("size", [2.0 ** e for e in (10, 20, 22, 23, 24, 25, 26, 27)])
def test_enormous_scores_in_an_8bit_cache(cuda_dev, size):
    """Scores so large that log2 of a value's scale is lost in them: the token far above the others has all the mass, and
    the output is its value, whatever its scale (the weight has to stay in fp16's range)."""
    hd, n = 64, 70
    g = torch.Generator("cpu").manual_seed(32)
    for e in (-9, -4, -1, 0, 1, 3, 6, 9):
        k, v = torch.zeros((n, hd)), torch.randint(-15, 16, (n, hd), generator=g).float() * 2.0 ** e / 8
        k[:, 0] = 0.5
        k[41, 0] = 1.0  # the others' scores are half of its
        out, lse, rl, ro, _, _ = _direct(cuda_dev, k, v, torch.ones(hd), size)
        assert ((out - ro).abs() <= 2.0 ** -8 * ro.abs() + 1e-30).all(), (size, e)
        assert abs(lse - rl) <= 2.0 ** -22 * rl + 2.0 ** -14
