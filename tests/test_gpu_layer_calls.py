"""How the operators around the FFN are called: from several threads, on other streams, in CUDA graphs. What is
computed is checked elsewhere; here every result is compared bit for bit with that of the plain call."""
import threading

import pytest
import torch

from activation_sparse_ffn_gate_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_dev):
    build.build()
    binding.load()
    binding.status_buffer(cuda_dev).zero_()
    yield
    assert binding.twell_read_status() == 0, "device status was raised"


def _rand(dev, *shape, seed, dtype=BF, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).to(dev)


class Attn:
    """An attention whose sequences are split over many blocks: parts in the workspace, joined by a second kernel."""

    def __init__(self, dev, seed, n=6000, B=2, hd=128):
        k, v = (_rand(dev, 40 * B, 2, 64, hd, seed=seed + i, dtype=F32).to(BF) for i in (0, 1))
        pages = -(-n // 64)
        self.cache = binding.KVCache(k, v)
        self.table = (torch.arange(B * pages, dtype=torch.int32, device=dev) % (40 * B)).view(B, pages)
        self.lens = torch.tensor([n - 13 * i for i in range(B)], dtype=torch.int32, device=dev)
        self.q = _rand(dev, B, 8, hd, seed=seed + 2)

    def __call__(self, **kw):
        return binding.twell_paged_attn_decode(self.q, self.cache, self.table, self.lens, **kw)[0]


class Grad:
    """A norm's backward: partial rows of dw in the workspace, added by a second kernel."""

    def __init__(self, dev, seed, N=900, d=1024):
        self.h, self.dy = _rand(dev, N, d, seed=seed, dtype=F32), _rand(dev, N, d, seed=seed + 1, dtype=F32)
        self.w = _rand(dev, d, seed=seed + 2, dtype=F32)
        self.rstd = torch.rsqrt(self.h.square().mean(-1) + 1e-6)

    def __call__(self, **kw):
        return torch.cat([t.reshape(-1) for t in
                          binding.twell_add_rmsnorm_bwd(self.dy, self.h, self.w, self.rstd, **kw)])


@pytest.mark.parametrize("what", [Attn, Grad])
def test_threads_that_share_a_stream(cuda_dev, what):
    """The default stream is the same for all threads, and so is its workspace; a call's two launches stay together."""
    calls = [what(cuda_dev, 10 * i) for i in range(6)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, errors = [[] for _ in calls], []
    start = threading.Barrier(len(calls))

    def run(i):
        try:
            start.wait()
            for _ in range(60):
                got[i].append(calls[i]())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert all(torch.equal(o, w) for os, w in zip(got, want) for o in os)


def _capture(call, stream):
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = call()
    return graph, out


@pytest.mark.parametrize("small,large", [(lambda dev: Grad(dev, 1, 400, 256), lambda dev: Grad(dev, 4, 4000, 8192)),
                                         (lambda dev: Attn(dev, 1, hd=64), lambda dev: Attn(dev, 4, hd=256))],
                         ids=["grad", "attn"])
def test_a_graph_writes_to_no_ones_memory(cuda_dev, small, large):
    """A larger call on the stream after the capture, then tensors that fill what the allocator has free: they keep their
    values through the replays, and the graph's results are the call's."""
    call, more = small(cuda_dev), large(cuda_dev)
    want = call()
    side = torch.cuda.Stream()
    graph, out = _capture(call, side)
    with torch.cuda.stream(side):
        more()
        side.synchronize()
        fills = [torch.full((n,), 7, dtype=torch.uint8, device=cuda_dev) for n in [1 << 20] * 40 + [1 << 22] * 20]
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((t == 7).all()) for t in fills)


@pytest.mark.parametrize("what", [Attn, Grad])
def test_a_graph_replays_beside_other_calls(cuda_dev, what):
    """Two graphs captured on one stream and plain calls on that stream, all at once on three streams."""
    a, b, c = (what(cuda_dev, 10 * i) for i in range(3))
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
    assert torch.equal(graphs[0][1], want[0]) and torch.equal(graphs[1][1], want[1])
    assert all(torch.equal(o, want[2]) for o in got)


def test_the_tensors_device_is_made_current(cuda_dev, monkeypatch):
    """With one device there is nothing else to be on: the quantiser, which sets the device in Python, is seen to do so. The
    other calls do it in the native module, whose call() takes the device and cannot be made without."""
    seen = []
    device = torch.cuda.device

    class Seen(device):
        def __enter__(self):
            seen.append(self.idx)
            return super().__enter__()

    monkeypatch.setattr(torch.cuda, "device", Seen)
    binding.twell_w4_quantize(_rand(cuda_dev, 16, 128, seed=1))
    assert seen == [cuda_dev.index]


def _owner(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not a tensor of the allocator's")


def _calls(dev):
    """Every call that allocates its outputs, by name: what it returns on a stream."""
    x, w = _rand(dev, 8, 512, seed=1), _rand(dev, 512, seed=2)
    x32 = x.float()
    rstd = torch.rsqrt(x32.square().mean(-1) + 1e-6)
    Wg, Wu, Wd = (_rand(dev, 512, 512, seed=s, scale=0.04) for s in (3, 4, 5))
    Wd16, Wd16t = binding.twell_convert_f16(Wd), binding.twell_convert_f16_transposed(Wd)
    xl = _rand(dev, 256, 512, seed=6)
    a = binding.twell_gate_pack(xl, Wg)
    G = torch.relu(_rand(dev, 256, 512, seed=7))
    cache = binding.KVCache.empty(2, 16, 2, 128, BF, dev)
    slots = torch.arange(4, dtype=torch.int32, device=dev)
    binding.twell_kv_append(cache, x.view(8, 4, 128)[:4, :2], x.view(8, 4, 128)[:4, 2:], slots)
    table, lens = torch.zeros((8, 1), dtype=torch.int32, device=dev), torch.full((8,), 4, dtype=torch.int32, device=dev)
    P = binding.twell_w4_quantize(Wg)
    y, ctx = binding.twell_hybrid_fwd(xl, Wg, Wu, Wd, 400, 256)
    return {
        "add_rmsnorm_fwd": lambda s: binding.twell_add_rmsnorm_fwd(x, w, x32, training=True, stream=s),
        "add_rmsnorm_fwd_q8": lambda s: (lambda r: (r[0].values, r[0].scale, *r[1:]))(
            binding.twell_add_rmsnorm_fwd_q8(x, w, x32, group=128, training=True, stream=s)),
        "add_rmsnorm_bwd": lambda s: binding.twell_add_rmsnorm_bwd(x32, x32, w, rstd, stream=s),
        "kv_gather": lambda s: binding.twell_kv_gather(cache, slots, stream=s),
        "paged_attn_decode": lambda s: binding.twell_paged_attn_decode(x.view(8, 4, 128), cache, table, lens, stream=s)[:1],
        "w4_quantize": lambda s: (lambda r: (r.words, r.scales))(binding.twell_w4_quantize(Wg, stream=s)),
        "w4_matvec": lambda s: [binding.twell_w4_matvec(x, P, stream=s)],
        "gate_pack": lambda s: (lambda r: (r.vals, r.idx, r.cnt))(binding.twell_gate_pack(xl, Wg, stream=s)),
        "ffn_fused_fwd": lambda s: [binding.twell_ffn_fused_fwd(xl, Wu, Wd, a, stream=s)],
        "ffn_fused_fwd_f16down": lambda s: [binding.twell_ffn_fused_fwd_f16down(xl, Wu, Wd16, a, stream=s)],
        "ffn_union_fwd": lambda s: [binding.twell_ffn_union_fwd(xl, Wu, Wd16t, a, stream=s)],
        "ffn_gate_union_fwd": lambda s: [binding.twell_ffn_gate_union_fwd(xl, Wg, Wu, Wd16t, stream=s)[0]],
        "ffn_tile_union_fwd": lambda s: [binding.twell_ffn_tile_union_fwd(xl, Wu, Wd16, a, stream=s)],
        "ffn_decode": lambda s: [binding.twell_ffn_decode(x, Wg, Wu, Wd, stream=s)[0]],
        "convert_f16": lambda s: [binding.twell_convert_f16(Wd, stream=s)],
        "convert_f16_transposed": lambda s: [binding.twell_convert_f16_transposed(Wd, stream=s)],
        "unpack": lambda s: [binding.twell_unpack(a, stream=s)],
        "column_activity": lambda s: [binding.twell_column_activity(a, stream=s)],
        "count_nonzeros": lambda s: [binding.twell_count_nonzeros(a, stream=s)],
        "gather_rows": lambda s: [binding.twell_gather_rows(Wg, slots, stream=s)],
        "pack_from_gate": lambda s: (lambda r: (r.vals, r.cnt))(binding.twell_pack_from_gate(G, stream=s)),
        "gate_gemm": lambda s: [binding.twell_gate_gemm(xl, Wg, stream=s)],
        "hybrid_route_from_gate": lambda s: [binding.twell_hybrid_route_from_gate(G, 400, 256, stream=s).cnt],
        "hybrid_fwd": lambda s: (lambda r: (r[0], r[1].a))(binding.twell_hybrid_fwd(xl, Wg, Wu, Wd, 400, 256, stream=s)),
        "hybrid_bwd": lambda s: binding.twell_hybrid_bwd(xl, Wg, Wu, Wd, ctx, y, stream=s),
    }


def test_what_a_call_allocates_belongs_to_its_stream(cuda_dev):
    """Outputs that a call allocates lie in the memory of the stream that it is given; a stream of another library's, a
    handle alone, will do."""
    calls = _calls(cuda_dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()

    class Handle:
        cuda_stream = s.cuda_stream

    for name, call in calls.items():
        for stream in (s, Handle()):
            outs = call(stream)
            s.synchronize()
            assert all(_owner(t) == s.cuda_stream for t in outs), name


def _claims(t, shape):
    """A tensor over t's memory that says it has that shape: what no call may take at its word."""
    types = {BF: "<i2", F32: "<f4", torch.int32: "<i4"}

    class Claim:
        __cuda_array_interface__ = {"shape": shape, "typestr": types[t.dtype], "data": (t.data_ptr(), False), "version": 2}

    out = torch.as_tensor(Claim(), device=t.device)
    return out.view(BF) if t.dtype == BF else out


def test_sizes_past_32_bits_are_refused(cuda_dev):
    """2^32 rows do not become none."""
    n = 1 << 32
    f, b, i = (torch.zeros(4096, dtype=t, device=cuda_dev) for t in (F32, BF, torch.int32))
    x, w, rstd = _claims(f, (n, 8)), f[:8], _claims(f, (n,))
    cache = binding.KVCache.empty(4, 16, 1, 64, BF, cuda_dev)
    k, slots = _claims(b, (n, 1, 64)), _claims(i, (n,))
    P = binding.twell_w4_quantize(_rand(cuda_dev, 16, 32, seed=1), 32)
    for call in (lambda: binding.twell_add_rmsnorm_fwd(x, w, y=x), lambda: binding.twell_add_rmsnorm_bwd(x, x, w, rstd, dx=x),
                 lambda: binding.twell_kv_append(cache, k, k, slots),
                 lambda: binding.twell_kv_gather(cache, slots, k_out=k, v_out=k),
                 lambda: binding.twell_paged_attn_decode(k, cache, _claims(i, (n, 1)), slots, out=k),
                 lambda: binding.twell_paged_attn_decode(b[:64].view(1, 1, 64), cache, _claims(i, (1, n)), i[:1]),
                 lambda: binding.twell_w4_matvec(_claims(b, (n, 32)), P, y=_claims(b, (n, 16))),
                 lambda: binding.twell_w4_quantize(_claims(b, (n, 32)), 32),
                 lambda: binding.KVCache(*(_claims(b, (n, 1, 16, 64)),) * 2)):
        with pytest.raises(ValueError):
            call()


def test_tensors_without_memory_raise(cuda_dev):
    """A tensor that stands for others (inside a vmap) has no address: the error comes before the interpreter's lock is
    given up."""
    k, q = _rand(cuda_dev, 2, 3, 2, 64, seed=1), _rand(cuda_dev, 2, 3, 4, 64, seed=2)
    cache = binding.KVCache.empty(2, 16, 2, 64, BF, cuda_dev)
    slots, table = (torch.zeros(n, dtype=torch.int32, device=cuda_dev) for n in ((3,), (3, 1)))
    out = torch.empty((3, 4, 64), dtype=BF, device=cuda_dev)
    for call, t in ((lambda t: binding.twell_kv_append(cache, t, t, slots), k),
                    (lambda t: binding.twell_paged_attn_decode(t, cache, table, slots, out=out), q)):
        with pytest.raises(RuntimeError):
            torch.vmap(call)(t)


def test_axes_of_one_may_have_any_stride(cuda_dev):
    """The stride of an axis of size one addresses nothing: one key head, one page, one token, one sequence."""
    def strange(t, axis):  # the same tensor with another stride there
        stride = list(t.stride())
        assert t.shape[axis] == 1
        stride[axis] = 3
        return t.as_strided(t.shape, stride)

    for dtype in (BF, torch.float8_e4m3fn):
        k, v = (_rand(cuda_dev, 3, 1, 64, seed=s) for s in (1, 2))
        slots = torch.arange(3, dtype=torch.int32, device=cuda_dev)
        table, lens = torch.zeros((3, 1), dtype=torch.int32, device=cuda_dev), slots + 1
        q = _rand(cuda_dev, 3, 1, 64, seed=3)
        got = []
        for odd in (False, True):
            c = binding.KVCache.empty(1, 16, 1, 64, dtype, cuda_dev)
            if odd:
                parts = [strange(t, 0) for t in (c.k, c.v)] + [None if s is None else strange(s, 0) for s in (c.k_scale, c.v_scale)]
                parts[1] = strange(parts[1], 1)  # of the values alone
                if dtype != BF:
                    parts[3] = strange(parts[3], 1)
                c = binding.KVCache(*parts)
                binding.twell_kv_append(c, strange(k, 1), v, slots)
                got.append(binding.twell_paged_attn_decode(strange(q, 1), c, table, lens)[0])
                one = binding.twell_paged_attn_decode(strange(q[:1], 0), c, table[:1], lens[:1])[0]
                assert torch.equal(one, got[0][:1])
            else:
                binding.twell_kv_append(c, k, v, slots)
                got.append(binding.twell_paged_attn_decode(q, c, table, lens)[0])
        assert torch.equal(*got)


def test_a_threads_first_call(cuda_dev):
    """A call may be the first thing that a thread does on the device."""
    x, Wg = _rand(cuda_dev, 200, 512, seed=1), _rand(cuda_dev, 1024, 512, seed=2, scale=0.04)
    want = binding.twell_gate_pack(x, Wg)
    torch.cuda.synchronize()
    got = []

    def run():
        try:
            got.append(binding.twell_gate_pack(x, Wg))
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert isinstance(got[0], binding.TwELL), got
    assert torch.equal(got[0].cnt, want.cnt) and torch.equal(binding.twell_unpack(got[0]), binding.twell_unpack(want))


class Ffn:
    """The FFN by one of its paths: several kernels over one workspace."""

    def __init__(self, dev, seed, N=8, path="decode", d=512, f=1024):
        # 3% to 4% of the units are kept: the walk's order is fixed as long as few rows are cut into items
        self.x = _rand(dev, N, d, seed=seed).abs()
        self.W = [_rand(dev, f, d, seed=seed + i, scale=d ** -0.5) for i in (1, 2, 3)]
        self.W[0] -= 0.1 * d ** -0.5
        self.more = {"union": {"Wd16t_s": binding.twell_convert_f16_transposed(self.W[2])},
                     "tile_union": {"Wd16_s": binding.twell_convert_f16(self.W[2])}}.get(path, {})
        self.path = path

    def __call__(self, **kw):
        return binding.ffn_forward(self.x, *self.W, path=self.path, **self.more, **kw)


PATHS = [("decode", 3, 16), ("walk", 200, 3000), ("union", 200, 3000), ("tile_union", 200, 3000)]


@pytest.mark.parametrize("path,N", [(p, n) for p, n, _ in PATHS])
def test_threads_that_share_a_stream_run_the_ffn(cuda_dev, path, N):
    test_threads_that_share_a_stream(cuda_dev, lambda dev, seed: Ffn(dev, seed, N, path))


@pytest.mark.parametrize("path,N,more", PATHS)
def test_a_graph_of_the_ffn_writes_to_no_ones_memory(cuda_dev, path, N, more):
    test_a_graph_writes_to_no_ones_memory(cuda_dev, lambda dev: Ffn(dev, 1, N, path), lambda dev: Ffn(dev, 9, more, path))


@pytest.mark.parametrize("path,N", [(p, n) for p, n, _ in PATHS])
def test_a_graph_of_the_ffn_replays_beside_other_calls(cuda_dev, path, N):
    test_a_graph_replays_beside_other_calls(cuda_dev, lambda dev, seed: Ffn(dev, seed, N, path))
