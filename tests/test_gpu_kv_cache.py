"""GPU parity of the paged key-value cache's write and read-back (twell_kv_append, twell_kv_gather): a bf16
cache holds copies; an e4m3 cache holds, bit for bit, the codes and scales of the definition (fp32:
scale = a / 448, code = value * (448 / a) to nearest even, a = max(|values|, 2^-60)), which are checked against
64 bits too: code * scale is within half an e4m3 step, 2^-4 of the value or 2^-10 scale, plus 2^-20 of
either for the two fp32 roundings."""
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


def _cache(dev, pages, ps, H, hd, dtype, layout="heads"):
    """A cache of zeros: pages of heads of tokens, of tokens of heads, or keys and values in one buffer."""
    def make(shape, perm, dt):
        return torch.zeros(shape, dtype=torch.uint8 if dt == E4 else dt, device=dev).view(dt).permute(perm)
    if layout == "heads":
        k, v = (make((pages, H, ps, hd), (0, 1, 2, 3), dtype) for _ in range(2))
    elif layout == "tokens":
        k, v = (make((pages, ps, H, hd), (0, 2, 1, 3), dtype) for _ in range(2))
    else:
        kv = make((pages, 2, H, ps, hd), (0, 1, 2, 3, 4), dtype)
        k, v = kv[:, 0], kv[:, 1]
    if dtype == BF:
        return binding.KVCache(k, v)
    if layout == "joint":
        s = torch.zeros((pages, 2, H, ps), dtype=F32, device=dev)
        return binding.KVCache(k, v, s[:, 0], s[:, 1])
    return binding.KVCache(k, v, *(torch.zeros((pages, H, ps), dtype=F32, device=dev) for _ in range(2)))


def _tokens(dev, n, H, hd, seed, fused):
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn((n, 3 * H, hd), generator=g)
    x *= torch.exp(2 * torch.randn((n, 3 * H, 1), generator=g))
    x = x.to(BF).to(dev)
    if fused:
        return x[:, H:2 * H], x[:, 2 * H:]
    return x[:, H:2 * H].contiguous(), x[:, 2 * H:].contiguous()


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _codes(t):
    # tensors on both sides: a division by a number may be turned into a product with its reciprocal
    a = t.float().abs().amax(-1).clamp_min(2.0 ** -60)
    top = torch.full_like(a, 448.0)
    return (t.float() * (top / a)[..., None]).to(E4), a / top


CASES = [(1, 1, 64, 16, "heads"), (5, 3, 96, 1, "heads"), (37, 4, 128, 8, "tokens"), (200, 5, 256, 64, "joint"),
         (64, 20, 128, 16, "heads"), (9, 1, 16, 32, "tokens"), (130, 2, 208, 128, "heads"), (40, 7, 64, 1024, "joint")]


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("n,H,hd,ps,layout", CASES)
def test_append_and_gather(cuda_dev, n, H, hd, ps, layout, dtype, fused):
    pages = n // ps + 3
    cache = _cache(cuda_dev, pages, ps, H, hd, dtype, layout)
    k, v = _tokens(cuda_dev, n, H, hd, 1, fused)
    g = torch.Generator("cpu").manual_seed(2)
    slots = torch.randperm(pages * ps, generator=g)[:n].to(torch.int32)
    if n > 4:
        slots[3] = -1
    slots = slots.to(cuda_dev)
    binding.twell_kv_append(cache, k, v, slots)
    assert binding.twell_read_status() == 0
    live = slots >= 0
    pg, off = slots[live].long() // ps, slots[live].long() % ps
    for t, c, sc in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        want = torch.zeros((pages, H, ps, hd), dtype=torch.uint8 if dtype == E4 else dtype, device=cuda_dev)
        if dtype == BF:
            want[pg, :, off] = t[live]
            assert torch.equal(_bits(c), _bits(want))
            continue
        q, s = _codes(t[live])
        want[pg, :, off] = q.view(torch.uint8)
        assert torch.equal(_bits(c), want)
        wsc = torch.zeros((pages, H, ps), dtype=F32, device=cuda_dev)
        wsc[pg, :, off] = s
        assert torch.equal(sc, wsc)
        x = t[live].double()
        err = (q.double() * s.double()[..., None] - x).abs()
        step = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s.double()[..., None])
        assert (err <= step * (1 + 2.0 ** -16)).all()

    # read back: other order, repeats, an empty slot
    idx = torch.cat([slots.flip(0), slots[:1], torch.tensor([-1], dtype=torch.int32, device=cuda_dev)])
    ko, vo = binding.twell_kv_gather(cache, idx)
    assert binding.twell_read_status() == 0
    src = torch.cat([torch.arange(n - 1, -1, -1), torch.tensor([0, 0])]).to(cuda_dev)
    for t, o in ((k, ko), (v, vo)):
        if dtype == BF:
            want = t[src].clone()
        else:
            q, s = _codes(t[src])
            want = (q.float() * s[..., None]).to(BF)
        want[idx < 0] = 0
        assert torch.equal(o, want)


def test_rows_of_zeros_tiny_and_not_finite_values(cuda_dev):
    cache = _cache(cuda_dev, 1, 16, 1, 64, E4)
    k = torch.zeros((5, 1, 64), dtype=BF, device=cuda_dev)
    k[1, 0, 3] = 2.0 ** -70  # under the smallest largest value: 448 2^-10 = 0.4375 is a code, so it is kept
    k[2, 0, :] = 2.0 ** -126  # 448 2^-66: a code of zero
    k[3, 0, 5], k[3, 0, 6] = float("nan"), 1.0
    k[4, 0, 5], k[4, 0, 6] = float("inf"), 1.0
    binding.twell_kv_append(cache, k, k, torch.arange(5, dtype=torch.int32, device=cuda_dev))
    ko, _ = binding.twell_kv_gather(cache, torch.arange(5, dtype=torch.int32, device=cuda_dev))
    assert torch.count_nonzero(ko[:3]) == 1 and ko[1, 0, 3] == 2.0 ** -70
    assert torch.isnan(ko[3, 0, 5]) and ko[3, 0, 6] == 1.0 and torch.isfinite(ko[3, 0, 7:]).all()
    assert torch.isnan(ko[4]).all()  # an infinite scale: the whole row is lost, the next ones are not
    assert binding.twell_read_status() == 0


def test_bad_slots_are_reported_and_skipped(cuda_dev):
    cache = _cache(cuda_dev, 2, 16, 2, 64, BF)
    k, v = _tokens(cuda_dev, 3, 2, 64, 5, False)
    slots = torch.tensor([32, 4, -2], dtype=torch.int32, device=cuda_dev)
    binding.twell_kv_append(cache, k, v, slots)
    assert binding.twell_read_status() == 5  # TWELL_ERR_DEVICE_CHECK
    assert torch.equal(cache.k[0, :, 4], k[1])
    assert torch.count_nonzero(cache.k) == torch.count_nonzero(k[1])
    ko, _ = binding.twell_kv_gather(cache, slots)
    assert binding.twell_read_status() == 5
    assert torch.equal(ko[1], k[1]) and torch.count_nonzero(ko[0]) == 0 and torch.count_nonzero(ko[2]) == 0


def test_offsets_past_32_bits(cuda_dev):
    """A cache of 2^32 + elements a kind: the last pages are reached, the first ones not touched."""
    ps, H, hd = 64, 8, 128
    pages = (1 << 32) // (ps * H * hd) + 2
    k, v = (torch.zeros((pages, H, ps, hd), dtype=torch.uint8, device=cuda_dev).view(E4) for _ in range(2))
    s = [torch.zeros((pages, H, ps), dtype=F32, device=cuda_dev) for _ in range(2)]
    cache = binding.KVCache(k, v, *s)
    kn, vn = _tokens(cuda_dev, 2, H, hd, 6, False)
    slots = torch.tensor([pages * ps - 1, (pages - 2) * ps], dtype=torch.int32, device=cuda_dev)
    binding.twell_kv_append(cache, kn, vn, slots)
    q, sc = _codes(kn)
    assert torch.equal(_bits(k[-1, :, -1]), _bits(q[0])) and torch.equal(s[0][-1, :, -1], sc[0])
    assert torch.equal(_bits(k[-2, :, 0]), _bits(q[1]))
    assert torch.count_nonzero(k[0].view(torch.uint8)) == 0
    ko, vo = binding.twell_kv_gather(cache, slots)
    qv, sv = _codes(vn)
    assert torch.equal(vo, (qv.float() * sv[..., None]).to(BF))
    assert binding.twell_read_status() == 0


def test_refusals(cuda_dev):
    cache = _cache(cuda_dev, 2, 16, 2, 64, BF)
    k, v = _tokens(cuda_dev, 3, 2, 64, 7, False)
    slots = torch.arange(3, dtype=torch.int32, device=cuda_dev)
    for bad in (lambda: binding.twell_kv_append(cache, k.float(), v, slots),
                lambda: binding.twell_kv_append(cache, k[:, :1], v, slots),
                lambda: binding.twell_kv_append(cache, k, v, slots.long()),
                lambda: binding.twell_kv_append(cache, k, v, slots[:2]),
                lambda: binding.twell_kv_append(cache, k.transpose(1, 2).contiguous().transpose(1, 2), v, slots),
                lambda: binding.twell_kv_gather(cache, slots, k_out=k.float()),
                lambda: binding.KVCache(cache.k, cache.v.float()),
                lambda: binding.KVCache(cache.k, cache.v[:1]),
                lambda: binding.KVCache(cache.k.transpose(2, 3), cache.v.transpose(2, 3)),
                lambda: binding.KVCache(cache.k.view(torch.uint8).view(E4), cache.v.view(torch.uint8).view(E4))):
        with pytest.raises(ValueError):
            bad()
    for shape in ((2, 2, 12, 64), (2, 2, 16, 72), (2, 2, 16, 512)):  # page size, head_dim
        c = binding.KVCache(*(torch.zeros(shape, dtype=BF, device=cuda_dev) for _ in range(2)))
        with pytest.raises(binding.TwellError) as e:
            binding.twell_kv_gather(c, slots)
        assert e.value.code == binding.TWELL_ERR_UNSUPPORTED
    binding.twell_kv_append(cache, k[:0], v[:0], slots[:0])
    assert binding.twell_kv_gather(cache, slots[:0])[0].shape == (0, 2, 64)
