"""Decode steps of one decoder layer at the widths of the 1.5B-like layer: prompts' keys, rotated, and values go into an
8-bit paged cache, then each step plans its tokens (pages, slots, positions) on the device and runs add + norm, 4-bit
projection with the sequences' adapters, rotation, cache write, attention, 4-bit projection, add + norm and the sparse FFN
for one new token per sequence. Random weights; prints the time of a step, call by call and as a CUDA graph.

    python examples/decode_layer.py [--seqs 8] [--prompt 4000] [--steps 16] [--adapters 4] [--rank 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from activation_sparse_ffn_gate_gb300 import binding, build, synthetic  # noqa: E402
from activation_sparse_ffn_gate_gb300.block import DecoderLayer  # noqa: E402


def make_layer(dev, d=2048, f=5632, heads=16, kv_heads=8, head_dim=128, adapters=0, rank=16, seed=0):
    L = synthetic.layer_1p5b(N=1)
    t = L.torch_inputs(dev)
    g = torch.Generator(dev).manual_seed(seed)

    def rand(*shape, scale):
        return (scale * torch.randn(shape, generator=g, device=dev)).to(torch.bfloat16)

    norm = torch.ones(d, dtype=torch.bfloat16, device=dev)
    w_qkv = binding.twell_w4_quantize(rand((heads + 2 * kv_heads) * head_dim, d, scale=d ** -0.5))
    w_out = binding.twell_w4_quantize(rand(d, heads * head_dim, scale=(heads * head_dim) ** -0.5))
    layer = DecoderLayer(norm, w_qkv, w_out, norm.clone(), t["Wg_s"], t["Wu_s"], t["Wd_s"], heads, kv_heads, head_dim,
                         rotary=binding.Rotary(binding.scaled_frequencies(head_dim)[0], head_dim, device=dev))
    if adapters:
        def adapter(k, n):
            return binding.Adapters(rand(adapters, rank, k, scale=k ** -0.5), rand(adapters, n, rank, scale=0.1),
                                    torch.ones(adapters, device=dev))
        layer.adapters_qkv = adapter(d, (heads + 2 * kv_heads) * head_dim)
        layer.adapters_out = adapter(heads * head_dim, d)
    return layer


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=4000)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--adapters", type=int, default=4, help="low-rank adapters, one a sequence in turn; 0: none")
    ap.add_argument("--rank", type=int, default=16)
    a = ap.parse_args()
    build.build()
    dev = torch.device("cuda:0")
    layer = make_layer(dev, adapters=a.adapters, rank=a.rank)
    page, most = 64, a.prompt + 2 * a.steps + 3
    per_seq = -(-most // page)
    cache = binding.KVCache.empty(a.seqs * per_seq, page, layer.n_kv_heads, layer.head_dim, torch.float8_e4m3fn, dev)
    pool = binding.PagePool.full(a.seqs * per_seq, page, dev)
    table = torch.zeros((a.seqs, per_seq), dtype=torch.int32, device=dev)
    lens = torch.zeros(a.seqs, dtype=torch.int32, device=dev)
    adapter = torch.arange(a.seqs, dtype=torch.int32, device=dev) % a.adapters if a.adapters else None

    # the prompts: their keys and values, as a prompt's fused projection leaves them
    plan = binding.twell_kv_plan(pool, table, lens, torch.full_like(lens, a.prompt), a.seqs * a.prompt)
    kv = torch.randn((a.seqs * a.prompt, 2 * layer.n_kv_heads, layer.head_dim), device=dev, dtype=torch.bfloat16)
    k, v = kv[:, :layer.n_kv_heads], kv[:, layer.n_kv_heads:]
    binding.twell_rope_fwd(k, None, plan.positions, layer.rotary, k)
    binding.twell_kv_append(cache, k, v, plan.slots)

    x = torch.randn((a.seqs, layer.attn_norm.numel()), device=dev, dtype=torch.bfloat16)
    one = torch.ones_like(lens)

    def step():  # one more token a sequence, so that token i is sequence i's (StepPlan.per_token is for other steps)
        p = binding.twell_kv_plan(pool, table, lens, one, a.seqs, labels=adapter)
        return layer.decode(x, None, cache, p.slots, table, lens, positions=p.positions,
                            adapter_ids=p.owner if a.adapters else None)

    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for name, run in (("call by call", step), ("as a CUDA graph", graph.replay)):
        spent = 0.0
        for _ in range(a.steps):
            start.record()
            run()
            end.record()
            torch.cuda.synchronize()
            spent += start.elapsed_time(end)
        print(f"{a.seqs} sequences of {a.prompt} tokens, one layer, {name}: {1000 * spent / a.steps:.1f} us a step")
    assert lens.tolist() == [a.prompt + 2 + 2 * a.steps] * a.seqs
    binding.check_device_status("decode")


if __name__ == "__main__":
    main()
