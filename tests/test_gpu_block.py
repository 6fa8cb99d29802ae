"""The decoder layer put together from the library's calls (block.py), on the GPU.

A step is checked against the same layer in 64 bits, with the weights that the 4-bit codes stand for and, for an e4m3
cache, the keys and values that its codes stand for. Seven tensors are rounded to bf16 on the way (two norms, the
fused projection, the attention's output, the output projection, the FFN's output; the FFN's inner h carries 11 bits or
more): each adds at most 2^-8 of its size, 2^-9.8 in the mean square, and the sublayers are near unit gain, so
0.01 in the Frobenius norm leaves a factor of about 3 over sqrt(7) 2^-9.8 = 0.003."""
import math

import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, block, build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
REL = 0.01


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()
    binding.status_buffer(cuda_dev).zero_()
    yield
    assert binding.twell_read_status() == 0, "device status was raised"


def _rand(dev, *shape, seed, scale=1.0, dtype=BF):
    g = torch.Generator("cpu").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).to(dev)


def _layer(dev, d, f, hq, hk, hd, group=64, rotate=None):
    return block.DecoderLayer(
        (1 + _rand(dev, d, seed=1, scale=0.1).float()).to(BF),
        binding.twell_w4_quantize(_rand(dev, (hq + 2 * hk) * hd, d, seed=2, scale=d ** -0.5), group),
        binding.twell_w4_quantize(_rand(dev, d, hq * hd, seed=3, scale=(hq * hd) ** -0.5), group),
        (1 + _rand(dev, d, seed=4, scale=0.1).float()).to(BF),
        _rand(dev, f, d, seed=5, scale=d ** -0.5), _rand(dev, f, d, seed=6, scale=d ** -0.5),
        _rand(dev, f, d, seed=7, scale=f ** -0.5), hq, hk, hd, rotate=rotate)


def _norm(h, w, eps):
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * w.double()


def _rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("cache_dtype", [BF, torch.float8_e4m3fn])
@pytest.mark.parametrize("hd,hq,hk,first", [(64, 8, 2, True), (128, 4, 4, False), (96, 6, 2, False)])
def test_decode_steps(cuda_dev, hd, hq, hk, first, cache_dtype):
    d, f, B, page = 512, 1024, 5, 16
    layer = _layer(cuda_dev, d, f, hq, hk, hd)
    lens = [0, 3, 16, 70, 200]
    cols = 16
    cache = binding.KVCache.empty(B * cols, page, hk, hd, cache_dtype, cuda_dev)
    table = torch.randperm(B * cols, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(B, cols).to(cuda_dev)
    past = [(_rand(cuda_dev, n, hk, hd, seed=20 + b), _rand(cuda_dev, n, hk, hd, seed=40 + b)) for b, n in enumerate(lens)]
    for b, (k, v) in enumerate(past):
        pos = torch.arange(lens[b], device=cuda_dev)
        slots = (table[b, pos // page] * page + pos % page).to(torch.int32)
        binding.twell_kv_append(cache, k, v, slots)
    for step in range(3):
        delta = _rand(cuda_dev, B, d, seed=60 + step)
        h = None if first else _rand(cuda_dev, B, d, seed=70 + step, dtype=torch.float32)
        pos = torch.tensor(lens, device=cuda_dev) + step
        rows = torch.arange(B, device=cuda_dev)
        slots = (table[rows, pos // page] * page + pos % page).to(torch.int32)
        now = (pos + 1).to(torch.int32)
        out, h2 = layer.decode(delta, h, cache, slots, table, now)
        # the layer in 64 bits; the keys and values as the cache holds them
        h1 = delta.double() + (h.double() if h is not None else 0.0)
        qkv = _norm(h1, layer.attn_norm, layer.eps) @ layer.w_qkv.dequantize().double().t()
        q = qkv[:, :hq * hd].view(B, hk, hq // hk, hd)
        a = torch.zeros((B, hk, hq // hk, hd), dtype=torch.float64, device=cuda_dev)
        for b in range(B):
            p = torch.arange(int(now[b]), device=cuda_dev)
            k, v = binding.twell_kv_gather(cache, (table[b, p // page] * page + p % page).to(torch.int32))
            z = torch.einsum("hgd,nhd->hgn", q[b], k.double()) / math.sqrt(hd)
            a[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), v.double())
        o = a.view(B, hq * hd) @ layer.w_out.dequantize().double().t()
        r2 = h1 + o
        y = _norm(r2, layer.ffn_norm, layer.eps)
        g = y @ layer.Wg_s.double().t()
        ref = (torch.relu(g) * (y @ layer.Wu_s.double().t())) @ layer.Wd_s.double()
        assert _rel(h2, r2) <= REL and _rel(out, ref) <= REL
        # the new tokens are in the cache: what the projection gave, to its type
        k, v = binding.twell_kv_gather(cache, slots)
        near = 2.0 ** -6 if cache_dtype == BF else 2.0 ** -4
        assert _rel(k, qkv[:, hq * hd:(hq + hk) * hd].view(B, hk, hd)) <= near
        assert _rel(v, qkv[:, (hq + hk) * hd:].view(B, hk, hd)) <= near


def test_rotation_is_applied_before_the_keys_are_stored(cuda_dev):
    seen = []

    def rotate(q, k):
        seen.append((q.shape, k.shape))
        k.neg_()

    hd, hq, hk = 64, 4, 2
    plain, turned = (_layer(cuda_dev, 256, 512, hq, hk, hd, rotate=r) for r in (None, rotate))
    table = torch.zeros((3, 1), dtype=torch.int32, device=cuda_dev)
    table[:, 0] = torch.arange(3)
    slots = torch.arange(3, dtype=torch.int32, device=cuda_dev) * 16
    lens = torch.ones(3, dtype=torch.int32, device=cuda_dev)
    x = _rand(cuda_dev, 3, 256, seed=80)
    keys = []
    for layer in (plain, turned):
        cache = binding.KVCache.empty(3, 16, hk, hd, BF, cuda_dev)
        layer.decode(x, None, cache, slots, table, lens)
        keys.append(binding.twell_kv_gather(cache, slots)[0])
    assert seen == [((3, hq, hd), (3, hk, hd))]
    assert torch.equal(keys[0], -keys[1])


def test_a_step_replays_in_a_cuda_graph(cuda_dev):
    hd, hq, hk, B, page = 128, 8, 2, 4, 64
    layer = _layer(cuda_dev, 512, 1024, hq, hk, hd)
    cache = binding.KVCache.empty(B * 40, page, hk, hd, torch.float8_e4m3fn, cuda_dev)
    table = torch.arange(B * 40, dtype=torch.int32, device=cuda_dev).view(B, 40)
    n = 2000
    pos = torch.arange(n, device=cuda_dev)
    for b in range(B):
        binding.twell_kv_append(cache, _rand(cuda_dev, n, hk, hd, seed=b), _rand(cuda_dev, n, hk, hd, seed=9 + b),
                                (table[b, pos // page] * page + pos % page).to(torch.int32))
    x = _rand(cuda_dev, B, 512, seed=90)
    lens = torch.full((B,), n + 1, dtype=torch.int32, device=cuda_dev)
    slots = (table[:, n // page] * page + n % page).to(torch.int32)
    out, h = layer.decode(x, None, cache, slots, table, lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        layer.decode(x, None, cache, slots, table, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        again, ha = layer.decode(x, None, cache, slots, table, lens)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(h, ha)
    # another length, the same graph
    lens.fill_(700)
    graph.replay()
    torch.cuda.synchronize()
    fresh, _ = layer.decode(x, None, cache, slots, table, lens)
    assert torch.equal(again, fresh)


def test_training_step_of_the_ffn_half(cuda_dev):
    """Forward and gradients against 64-bit autograd, the FFN's from its own input: the norm's output as it was rounded to
    bf16 (against the unrounded one, a gate entry within that rounding of zero changes sides in about 4e-4 of the
    places, and a gradient moves by the root of that, 2%, whatever is computed). The FFN's gradients are held to 5e-3
    (tests/parity.py); the norm's pass on what they are given with an error of fp32, so the same bound holds
    behind it."""
    N, d, f, K = 96, 256, 512, 300
    h, delta = _rand(cuda_dev, N, d, seed=1, dtype=torch.float32, scale=2.0), _rand(cuda_dev, N, d, seed=2)
    w = (1 + _rand(cuda_dev, d, seed=3, scale=0.1).float()).to(BF)
    Wg, Wu = (_rand(cuda_dev, f, d, seed=s, scale=d ** -0.5) for s in (4, 5))
    Wd = _rand(cuda_dev, f, d, seed=6, scale=f ** -0.5)
    df, dh = _rand(cuda_dev, N, d, seed=7), _rand(cuda_dev, N, d, seed=8, dtype=torch.float32)
    out, h1, saved = block.ffn_sublayer_fwd(delta, h, w, Wg, Wu, Wd, K, N, l1_coef=0.0)
    y = saved[0]
    grads = block.ffn_sublayer_bwd(df, dh, saved)
    r, wn = (delta.double() + h.double()).requires_grad_(), w.double().requires_grad_()
    norm = r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6) * wn
    assert _rel(h1, r.detach()) <= 1e-6 and _rel(y, norm.detach()) <= 2.0 ** -8
    P = [t.double().requires_grad_() for t in (y, Wg, Wu, Wd)]
    ref = (torch.relu(P[0] @ P[1].t()) * (P[0] @ P[2].t())) @ P[3]
    assert _rel(out, ref.detach()) <= 5e-3
    (ref * df.double()).sum().backward()
    ((norm * P[0].grad).sum() + (r * dh.double()).sum()).backward()
    for got, want in zip(grads, (r.grad, wn.grad, P[1].grad, P[2].grad, P[3].grad)):
        assert got.dtype == torch.float32 and _rel(got, want) <= 5e-3


def _busy(dev):
    """Allocations and fills on the current stream, as a program makes them beside another stream's work."""
    return [torch.full((n,), 3.0, dtype=BF, device=dev) for n in (256, 1024, 4096, 16384, 65536) for _ in range(20)]


@pytest.mark.parametrize("first", [True, False])
def test_decode_on_another_stream(cuda_dev, first):
    """A step with stream=s gives, bit for bit, what it gives on the current stream: the rotation is queued on s, and what
    the current stream allocates and fills meanwhile is none of the step's memory."""
    def rotate(q, k):
        seen.append(torch.cuda.current_stream())
        q.mul_(-0.5)
        k.mul_(2.0)

    seen = []
    hd, hq, hk, B, n = 128, 8, 2, 6, 300
    layer = _layer(cuda_dev, 512, 1024, hq, hk, hd, rotate=rotate)
    table = torch.arange(B * 5, dtype=torch.int32, device=cuda_dev).view(B, 5)
    past = [_rand(cuda_dev, B * n, hk, hd, seed=s) for s in (1, 2)]
    pos = torch.arange(n, device=cuda_dev)
    slots = (table[:, pos // 64] * 64 + pos % 64).to(torch.int32).reshape(-1)
    new = (table[:, n // 64] * 64 + n % 64).to(torch.int32)
    lens = torch.full((B,), n + 1, dtype=torch.int32, device=cuda_dev)
    x = _rand(cuda_dev, B, 512, seed=91)
    h = None if first else _rand(cuda_dev, B, 512, seed=92, dtype=torch.float32)

    def steps(stream):
        cache = binding.KVCache.empty(B * 5, 64, hk, hd, BF, cuda_dev)
        binding.twell_kv_append(cache, *past, slots)
        torch.cuda.synchronize()
        outs, other = [], []
        for _ in range(8):
            outs.append(layer.decode(x, h, cache, new, table, lens, stream=stream))
            other += _busy(cuda_dev)
        torch.cuda.synchronize()
        return outs, other

    want, _ = steps(None)
    s = torch.cuda.Stream()
    seen.clear()
    got, other = steps(s)
    assert seen == [s] * 8
    for (a, b), (c, d) in zip(got, want):
        assert torch.equal(a, c) and torch.equal(b, d)
    assert all(bool((t == 3.0).all()) for t in other)


def test_training_step_on_another_stream(cuda_dev):
    N, d, f, K = 64, 256, 512, 300
    h, delta = _rand(cuda_dev, N, d, seed=1, dtype=torch.float32, scale=2.0), _rand(cuda_dev, N, d, seed=2)
    w = (1 + _rand(cuda_dev, d, seed=3, scale=0.1).float()).to(BF)
    Wg, Wu = (_rand(cuda_dev, f, d, seed=s, scale=d ** -0.5) for s in (4, 5))
    Wd = _rand(cuda_dev, f, d, seed=6, scale=f ** -0.5)
    df, dh = _rand(cuda_dev, N, d, seed=7), _rand(cuda_dev, N, d, seed=8, dtype=torch.float32)

    def step(stream):
        torch.cuda.synchronize()
        out, h1, saved = block.ffn_sublayer_fwd(delta, h, w, Wg, Wu, Wd, K, N, stream=stream)
        other = _busy(cuda_dev)
        grads = block.ffn_sublayer_bwd(df, dh, saved, stream=stream)
        other += _busy(cuda_dev)
        torch.cuda.synchronize()
        assert all(bool((t == 3.0).all()) for t in other)
        return out, h1, grads[0], grads[1]

    want = step(None)
    for a, b in zip(step(torch.cuda.Stream()), want):
        assert torch.equal(a, b)


def test_training_step_without_a_stream_before_it(cuda_dev):
    """h None, as in DecoderLayer.decode: the stream is delta itself, forward and backward."""
    N, d, f, K = 64, 256, 512, 300
    delta, w = _rand(cuda_dev, N, d, seed=2), (1 + _rand(cuda_dev, d, seed=3, scale=0.1).float()).to(BF)
    Wg, Wu = (_rand(cuda_dev, f, d, seed=s, scale=d ** -0.5) for s in (4, 5))
    Wd = _rand(cuda_dev, f, d, seed=6, scale=f ** -0.5)
    df, dh = _rand(cuda_dev, N, d, seed=7), _rand(cuda_dev, N, d, seed=8, dtype=torch.float32)
    out = []
    for h in (None, torch.zeros_like(delta)):
        f_out, h1, saved = block.ffn_sublayer_fwd(delta, h, w, Wg, Wu, Wd, K, N)
        out.append((f_out, h1, *block.ffn_sublayer_bwd(df, dh, saved)))
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_a_step_on_another_librarys_stream(cuda_dev):
    """A stream that is a handle alone, as every call takes it."""
    s = torch.cuda.Stream()

    class Handle:
        cuda_stream = s.cuda_stream

    layer = _layer(cuda_dev, 256, 512, 4, 2, 64)
    table = torch.arange(3, dtype=torch.int32, device=cuda_dev)[:, None].contiguous()
    slots, lens = table[:, 0] * 16, torch.ones(3, dtype=torch.int32, device=cuda_dev)
    x = _rand(cuda_dev, 3, 256, seed=80)
    outs = []
    for stream in (None, Handle()):
        cache = binding.KVCache.empty(3, 16, 2, 64, BF, cuda_dev)
        torch.cuda.synchronize()
        outs.append(layer.decode(x, None, cache, slots, table, lens, stream=stream)[0])
        torch.cuda.synchronize()
    assert torch.equal(*outs)
