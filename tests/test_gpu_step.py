"""A served step as it is used: the plan, the rotation and the adapters with the decoder layer's other calls, call by call
and in CUDA graphs, on other streams and from several threads."""
import math
import threading

import pytest
import torch
from test_gpu_block import REL, _layer, _norm, _rand, _rel

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


def _adapters(dev, L, R, k, n, seed):
    return binding.Adapters(_rand(dev, L, R, k, seed=seed, scale=k ** -0.5), _rand(dev, L, n, R, seed=seed + 1, scale=0.5 * R ** -0.5),
                            torch.linspace(0.5, 1.5, L, device=dev))


def _served(dev, d, f, hq, hk, hd, scaling="none"):
    layer = _layer(dev, d, f, hq, hk, hd)
    freq, factor = binding.scaled_frequencies(hd, 10000.0, scaling, 4.0, original=64)
    layer.rotary = binding.Rotary(freq, hd, factor=factor)
    layer.adapters_qkv = _adapters(dev, 3, 16, d, (hq + 2 * hk) * hd, 90)
    layer.adapters_out = _adapters(dev, 3, 8, hq * hd, d, 95)
    return layer, torch.tensor(freq, dtype=torch.float64, device=dev), factor


def _turn(x, pos, freq, factor):
    t = pos.double()[:, None, None] * freq
    a, b = x[..., :len(freq)], x[..., len(freq):]
    return factor * torch.cat([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()], -1)


def _adapted(x, ad, ids):
    out = []
    for row, i in zip(x, ids.tolist()):
        out.append(torch.zeros(ad.b.shape[1], dtype=torch.float64, device=x.device) if i < 0 else
                   float(ad.scale[i]) * (ad.b[i].double() @ (ad.a[i].double() @ row)))
    return torch.stack(out)


@pytest.mark.parametrize("cache_dtype", [BF, torch.float8_e4m3fn])
@pytest.mark.parametrize("hd,hq,hk,scaling", [(64, 8, 2, "none"), (128, 4, 4, "ramp")])
def test_a_served_life(cuda_dev, hd, hq, hk, scaling, cache_dtype):
    """Prompts in one plan, then decode steps, an end and a new request in its row, each against 64 bits. Two more tensors are
    rounded to bf16 than in the layer's own test (the adapters' outputs, the turned heads): its bound holds nine."""
    d, f, B, page, cols = 512, 1024, 5, 16, 20
    layer, freq, factor = _served(cuda_dev, d, f, hq, hk, hd, scaling)
    pool = binding.PagePool.full(B * cols, page, cuda_dev)
    cache = binding.KVCache.empty(B * cols, page, hk, hd, cache_dtype, cuda_dev)
    table = torch.full((B, cols), -1, dtype=I32, device=cuda_dev)
    lens = torch.zeros(B, dtype=I32, device=cuda_dev)
    labels = torch.tensor([0, 2, -1, 1, 0], dtype=I32, device=cuda_dev)
    t = lambda v: torch.tensor(v, dtype=I32, device=cuda_dev)  # noqa: E731

    def bring(new, seed):  # prompts: their keys, turned, and values
        n = sum(max(x, 0) for x in new)
        p = binding.twell_kv_plan(pool, table, lens, t(new), n + 3)
        k, v = (_rand(cuda_dev, n + 3, hk, hd, seed=seed + i) for i in (0, 1))
        binding.twell_rope_fwd(k, None, p.positions, layer.rotary, k)
        binding.twell_kv_append(cache, k, v, p.slots)

    bring([3, 17, 1, 70, 200], 20)
    W, Wo = layer.w_qkv.dequantize().double(), layer.w_out.dequantize().double()
    for step in range(4):
        if step == 2:  # the fourth request has ended, and another comes into its row
            before = lens.tolist()
            bring([0, 0, 0, -1, 0], 30)
            assert lens.tolist() == before[:3] + [0] + before[4:]
            bring([0, 0, 0, 33, 0], 40)
        delta, h = _rand(cuda_dev, B, d, seed=60 + step), _rand(cuda_dev, B, d, seed=70 + step, dtype=F32)
        p = binding.twell_kv_plan(pool, table, lens, torch.ones_like(lens), B, labels=labels)
        assert torch.equal(p.owner, labels) and torch.equal(p.positions, lens - 1)
        out, h2 = layer.decode(delta, h, cache, p.slots, table, lens, positions=p.positions, adapter_ids=p.owner)
        h1 = delta.double() + h.double()
        y = _norm(h1, layer.attn_norm, layer.eps)
        qkv = (y @ W.t() + _adapted(y, layer.adapters_qkv, labels)).view(B, hq + 2 * hk, hd)
        q = _turn(qkv[:, :hq], p.positions, freq, factor).view(B, hk, hq // hk, hd)
        a = torch.zeros((B, hk, hq // hk, hd), dtype=torch.float64, device=cuda_dev)
        for b in range(B):
            at = torch.arange(int(lens[b]), device=cuda_dev)
            k, v = binding.twell_kv_gather(cache, (table[b, at // page] * page + at % page).to(I32))
            z = torch.einsum("hgd,nhd->hgn", q[b], k.double()) / math.sqrt(hd)
            a[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), v.double())
        a = a.view(B, hq * hd)
        r2 = h1 + a @ Wo.t() + _adapted(a, layer.adapters_out, labels)
        y = _norm(r2, layer.ffn_norm, layer.eps)
        ref = (torch.relu(y @ layer.Wg_s.double().t()) * (y @ layer.Wu_s.double().t())) @ layer.Wd_s.double()
        assert _rel(h2, r2) <= REL and _rel(out, ref) <= REL
        k, _ = binding.twell_kv_gather(cache, p.slots)
        near = 2.0 ** -6 if cache_dtype == BF else 2.0 ** -4
        assert _rel(k, _turn(qkv[:, hq:hq + hk], p.positions, freq, factor)) <= near
    held = sum(-(-n // page) for n in lens.tolist())
    assert pool.state[1].item() == B * cols - held


def test_a_layer_without_them_is_what_it_was(cuda_dev):
    layer = _layer(cuda_dev, 256, 512, 4, 2, 64)
    x = _rand(cuda_dev, 3, 256, seed=80)
    slots, lens = torch.arange(3, dtype=I32, device=cuda_dev) * 16, torch.ones(3, dtype=I32, device=cuda_dev)
    table = torch.arange(3, dtype=I32, device=cuda_dev).view(3, 1)
    cache = lambda: binding.KVCache.empty(3, 16, 2, 64, BF, cuda_dev)  # noqa: E731
    want = layer.decode(x, None, cache(), slots, table, lens)
    none = torch.full((3,), -1, dtype=I32, device=cuda_dev)
    layer.adapters_qkv, layer.adapters_out = _adapters(cuda_dev, 2, 8, 256, 512, 1), _adapters(cuda_dev, 2, 8, 256, 256, 3)
    layer.rotary = binding.Rotary([1.0] * 32, 64)
    got = layer.decode(x, None, cache(), slots, table, lens, positions=slots * 0, adapter_ids=none)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(ValueError):
        layer.decode(x, None, cache(), slots, table, lens)


def test_steps_replay_in_a_cuda_graph(cuda_dev):
    """A whole step in one graph, plan and all: its replays go on token by token, as calls do."""
    d, B, page, cols = 256, 4, 4, 8
    layer, _, _ = _served(cuda_dev, d, 512, 4, 2, 64)
    x = _rand(cuda_dev, B, d, seed=81)
    labels = torch.tensor([1, -1, 0, 2], dtype=I32, device=cuda_dev)
    ones = torch.ones(B, dtype=I32, device=cuda_dev)

    def world():
        return (binding.PagePool.full(B * cols, page, cuda_dev), binding.KVCache.empty(B * cols, page, 2, 64, BF, cuda_dev),
                torch.full((B, cols), -1, dtype=I32, device=cuda_dev), torch.zeros(B, dtype=I32, device=cuda_dev))

    def step(pool, cache, table, lens):
        p = binding.twell_kv_plan(pool, table, lens, ones, B, labels=labels)
        return layer.decode(x, None, cache, p.slots, table, lens, positions=p.positions, adapter_ids=p.owner)

    w = world()
    want = [[t.clone() for t in step(*w)] for _ in range(10)]
    v = world()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(*world())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(*v)
    for i in range(10):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
    assert torch.equal(v[2], w[2]) and torch.equal(v[3], w[3]) and torch.equal(v[0].state, w[0].state)


class Lora:
    """An adapters' call whose kernels leave something in the workspace for one another."""

    def __init__(self, dev, seed, N=1100, k=128, n=136, L=5):
        self.ad = _adapters(dev, L, 16, k, n, seed)
        self.x, self.y = _rand(dev, N, k, seed=seed + 3), _rand(dev, N, n, seed=seed + 4)
        self.ids = (torch.arange(N, device=dev) * (seed + 7) % (L + 1) - 1).to(I32)

    def __call__(self, **kw):
        return binding.twell_lora_add(self.y, self.x, self.ad, self.ids, out=torch.empty_like(self.y), **kw)


def _capture(call, stream):
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = call()
    return graph, out


@pytest.mark.parametrize("sizes", [[(700 + 311 * i, 5) for i in range(5)], [(60 + 90 * i, 50) for i in range(5)]], ids=["grouped", "found"])
def test_threads_that_share_a_stream(cuda_dev, sizes):
    calls = [Lora(cuda_dev, 10 * i, N=N, L=L) for i, (N, L) in enumerate(sizes)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, errors, start = [[] for _ in calls], [], threading.Barrier(len(calls))

    def run(i):
        try:
            start.wait()
            for _ in range(50):
                got[i].append(calls[i]())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not errors and all(torch.equal(o, w) for os, w in zip(got, want) for o in os)


@pytest.mark.parametrize("sizes", [[(900, 5), (1400, 5), (1900, 5)], [(64, 64), (200, 40), (500, 30)], [(3, 5), (16, 9), (100, 2)]],
                         ids=["grouped", "found", "whole"])
def test_graphs_beside_calls(cuda_dev, sizes):
    """Two graphs captured on one stream and plain calls on it, at once on three streams; then tensors that fill what the
    allocator has free keep their values through the replays."""
    a, b, c = (Lora(cuda_dev, 10 * i, N=N, L=L) for i, (N, L) in enumerate(sizes))
    want = [x() for x in (a, b, c)]
    side, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    graphs = [_capture(x, side) for x in (a, b)]
    got = []
    for _ in range(30):
        for (g, _), s in zip(graphs, others):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(side):
            got.append(c())
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want[0]) and torch.equal(graphs[1][1], want[1]) and all(torch.equal(o, want[2]) for o in got)
    with torch.cuda.stream(side):
        fills = [torch.full((n,), 7, dtype=torch.uint8, device=cuda_dev) for n in [1 << 20] * 40 + [1 << 22] * 20]
    torch.cuda.synchronize()
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in fills) and torch.equal(graphs[0][1], want[0])


@pytest.mark.parametrize("N,L", [(1100, 5), (64, 64), (4, 5)])
def test_a_workspace_of_the_callers(cuda_dev, N, L):
    call = Lora(cuda_dev, 3, N=N, L=L)
    n = binding.twell_workspace_bytes(binding.OP_LORA_ADD, call.x.shape[0], call.ad.a.shape[1], 1)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device=cuda_dev)  # its contents do not matter
    assert torch.equal(call(ws=ws), call())


def _owner(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not a tensor of the allocator's")


def test_what_a_call_allocates_belongs_to_its_stream(cuda_dev):
    q = _rand(cuda_dev, 6, 4, 64, seed=1)
    pos = torch.arange(6, dtype=I32, device=cuda_dev)
    r = binding.Rotary([1.0] * 32, 64)
    table, lens = torch.zeros((2, 4), dtype=I32, device=cuda_dev), torch.zeros(2, dtype=I32, device=cuda_dev)
    calls = {"rope_fwd": lambda s: binding.twell_rope_fwd(q, q, pos, r, stream=s),
             "rope_bwd": lambda s: binding.twell_rope_bwd(q, q, pos, r, stream=s),
             "kv_plan": lambda s: (lambda p: (p.slots, p.positions, p.owner, p.starts))(
                 binding.twell_kv_plan(binding.PagePool.full(8, 16, cuda_dev), table, lens, lens + 1, 4, stream=s))}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()

    class Handle:
        cuda_stream = s.cuda_stream

    for name, call in calls.items():
        for stream in (s, Handle()):
            torch.cuda.synchronize()
            outs = call(stream)
            s.synchronize()
            assert all(_owner(t) == s.cuda_stream for t in outs), name
    lora = Lora(cuda_dev, 2)
    out = torch.empty_like(lora.y)
    torch.cuda.synchronize()
    binding.twell_lora_add(lora.y, lora.x, lora.ad, lora.ids, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, lora())


def _claims(t, shape):
    """A tensor over t's memory that says it has that shape: what no call may take at its word."""
    types = {BF: "<i2", F32: "<f4", I32: "<i4"}

    class Claim:
        __cuda_array_interface__ = {"shape": shape, "typestr": types[t.dtype], "data": (t.data_ptr(), False), "version": 2}

    out = torch.as_tensor(Claim(), device=t.device)
    return out.view(BF) if t.dtype == BF else out


def test_sizes_past_32_bits_are_refused(cuda_dev):
    n = 1 << 32
    b, i = (torch.zeros(4096, dtype=t, device=cuda_dev) for t in (BF, I32))
    r = binding.Rotary([1.0] * 4, 8)
    pool = binding.PagePool.full(8, 16, cuda_dev)
    ad = binding.Adapters(_claims(b, (2, 8, 8)), _claims(b, (2, 8, 8)), torch.ones(2, device=cuda_dev))
    for call in (lambda: binding.twell_rope_fwd(_claims(b, (n, 1, 8)), None, _claims(i, (n,)), r, _claims(b, (n, 1, 8))),
                 lambda: binding.twell_rope_fwd(_claims(b, (n, 1, 1, 8)), None, _claims(i, (1,)), r, _claims(b, (n, 1, 1, 8))),
                 lambda: binding.twell_kv_plan(pool, _claims(i, (1, n)), i[:1], i[:1], 4),
                 lambda: binding.twell_kv_plan(pool, _claims(i, (1, 4)), i[:1], i[:1], n),
                 lambda: binding.twell_lora_add(_claims(b, (n, 8)), _claims(b, (n, 8)), ad, _claims(i, (n,)))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: binding.twell_rope_fwd(_claims(b, (1 << 28, 1, 8)), None, _claims(i, (1 << 28,)), r, _claims(b, (1 << 28, 1, 8))),
                 lambda: binding.twell_lora_add(*(_claims(b, ((1 << 20) + 1, 8)),) * 2, ad, _claims(i, ((1 << 20) + 1,)))):
        with pytest.raises(binding.TwellError) as e:
            call()
        assert e.value.code == binding.TWELL_ERR_UNSUPPORTED


def test_tensors_without_memory_raise(cuda_dev):
    q = _rand(cuda_dev, 2, 3, 2, 64, seed=1)
    pos = torch.zeros(3, dtype=I32, device=cuda_dev)
    r = binding.Rotary([1.0] * 32, 64)
    lora = Lora(cuda_dev, 2, N=3)
    out = torch.empty((3, 2, 64), dtype=BF, device=cuda_dev)
    for call, t in ((lambda t: binding.twell_rope_fwd(t, None, pos, r, out)[0], q),
                    (lambda t: binding.twell_lora_add(lora.y, t, lora.ad, lora.ids), torch.stack([lora.x, lora.x]))):
        with pytest.raises(RuntimeError):
            torch.vmap(call)(t)
    torch.cuda.synchronize()
