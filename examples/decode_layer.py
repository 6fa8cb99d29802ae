"""Decode steps of one decoder layer at the widths of the 1.5B-like layer: prompts' keys and values go into an 8-bit
paged cache, then each step runs add + norm, 4-bit projection, cache write, attention, 4-bit projection, add +
norm and the sparse FFN for one new token per sequence. Random weights; prints the time of a step, call by call
and as a CUDA graph.

    python examples/decode_layer.py [--seqs 8] [--prompt 4000] [--steps 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from activation_sparse_ffn_gate_gb300 import binding, build, synthetic  # noqa: E402
from activation_sparse_ffn_gate_gb300.block import DecoderLayer  # noqa: E402


def make_layer(dev, d=2048, f=5632, heads=16, kv_heads=8, head_dim=128, seed=0):
    L = synthetic.layer_1p5b(N=1)
    t = L.torch_inputs(dev)
    g = torch.Generator(dev).manual_seed(seed)

    def rand(*shape, scale):
        return (scale * torch.randn(shape, generator=g, device=dev)).to(torch.bfloat16)

    norm = torch.ones(d, dtype=torch.bfloat16, device=dev)
    w_qkv = binding.twell_w4_quantize(rand((heads + 2 * kv_heads) * head_dim, d, scale=d ** -0.5))
    w_out = binding.twell_w4_quantize(rand(d, heads * head_dim, scale=(heads * head_dim) ** -0.5))
    return DecoderLayer(norm, w_qkv, w_out, norm.clone(), t["Wg_s"], t["Wu_s"], t["Wd_s"], heads, kv_heads, head_dim)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=4000)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    build.build()
    dev = torch.device("cuda:0")
    layer = make_layer(dev)
    page, most = 64, a.prompt + a.steps
    per_seq = -(-most // page)
    cache = binding.KVCache.empty(a.seqs * per_seq, page, layer.n_kv_heads, layer.head_dim, torch.float8_e4m3fn, dev)
    table = torch.randperm(a.seqs * per_seq, device=dev).to(torch.int32).view(a.seqs, per_seq).contiguous()

    def slots_of(pos):  # slots of positions [seqs, n]
        return (torch.gather(table, 1, (pos // page).long()) * page + pos % page).to(torch.int32).reshape(-1)

    # the prompts: their keys and values, as a prompt's fused projection leaves them
    pos = torch.arange(a.prompt, device=dev).expand(a.seqs, -1)
    kv = torch.randn((a.seqs * a.prompt, 2 * layer.n_kv_heads, layer.head_dim), device=dev, dtype=torch.bfloat16)
    binding.twell_kv_append(cache, kv[:, :layer.n_kv_heads], kv[:, layer.n_kv_heads:], slots_of(pos))

    x = torch.randn((a.seqs, layer.attn_norm.numel()), device=dev, dtype=torch.bfloat16)
    lens = torch.full((a.seqs,), a.prompt, dtype=torch.int32, device=dev)
    slots = torch.zeros(a.seqs, dtype=torch.int32, device=dev)

    def step():
        return layer.decode(x, None, cache, slots, table, lens)

    def advance():  # the next token's slot, and the length that counts it
        slots.copy_(slots_of(lens[:, None]))
        lens.add_(1)

    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    advance()
    step()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for name, run in (("call by call", step), ("as a CUDA graph", graph.replay)):
        lens.fill_(a.prompt)
        spent = 0.0
        for _ in range(a.steps):
            advance()
            start.record()
            run()
            end.record()
            torch.cuda.synchronize()
            spent += start.elapsed_time(end)
        print(f"{a.seqs} sequences of {a.prompt} tokens, one layer, {name}: {1000 * spent / a.steps:.1f} us a step")
    binding.check_device_status("decode")


if __name__ == "__main__":
    main()
