"""One decoder layer served in 8 bits: prompts of several requests, then tokens.

    python examples/decoder_layer.py [--format mxfp8|fp8|fp8_block] [--prompts 700,33,1] [--tokens 32]

The layer's calls, in order (random weights; no positional encoding, which would go between the
qkv projection and the cache):

    rms_norm_operand   norm of the residual stream, quantized in the next layer's operand order
    linear_fused       q, k, v projections in one product
    kv_append          the new keys and values into the paged 8-bit cache
    attention_kv8      softmax attention over it
    linear_fused       output projection
    rms_norm_operand   adds it onto the residual stream, norm, quantized
    linear_fused       gate and up projections with silu(gate) * up in the epilogue
    linear_fused       down projection, the residual stream added in the epilogue

Prompts of different lengths run in one call without padding (cu_seqlens). The step for single
tokens has fixed shapes, so it is captured once in a HIP graph and replayed while the lengths, on
the device, grow.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import fp8_quantized_linear_amd as fql  # noqa: E402

X_SCALE = 0.1  # static activation scale of per-tensor FP8


def make_weight(fmt, N, K, gen, W=None):
    if W is None:
        W = torch.randn(N, K, generator=gen) * K ** -0.5
    W = W.cuda()
    if fmt == "fp8":
        return fql.FP8Weight.from_float(W, X_SCALE)
    return (fql.FP8BlockWeight if fmt == "fp8_block" else fql.MXFP8Weight).from_float(W)


class DecoderLayer:
    def __init__(self, fmt, hidden, q_heads, kv_heads, head_dim, ff, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.fmt, self.q_heads, self.kv_heads, self.head_dim = fmt, q_heads, kv_heads, head_dim
        self.qkv = make_weight(fmt, (q_heads + 2 * kv_heads) * head_dim, hidden, gen)
        self.o = make_weight(fmt, hidden, q_heads * head_dim, gen)
        gate, up = (torch.randn(ff, hidden, generator=gen) * hidden ** -0.5 for _ in range(2))
        self.gate_up = make_weight(fmt, 2 * ff, hidden, gen, fql.interleave_gate_up(gate, up))
        self.down = make_weight(fmt, hidden, ff, gen)
        self.norm1, self.norm2 = ((1 + 0.1 * torch.randn(hidden, generator=gen)).to(torch.bfloat16).cuda()
                                  for _ in range(2))
        self.scale = X_SCALE if fmt == "fp8" else None

    def __call__(self, h, cache, block_table, lens, cu_seqlens, max_new):
        """h: bf16 [tokens, hidden], the new tokens of all sequences one after the other."""
        x, _ = fql.rms_norm_operand(h, self.norm1, self.fmt, scale=self.scale)
        qkv = fql.linear_fused(x, self.qkv).unflatten(1, (-1, self.head_dim))
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        fql.kv_append(cache, k, v, block_table, lens, cu_seqlens, max_new)
        a = fql.attention_kv8(q, cache, block_table, lens, cu_seqlens, max_new)
        y = fql.linear_fused(a.flatten(1), self.o)
        x, h = fql.rms_norm_operand(y, self.norm2, self.fmt, residual=h, scale=self.scale)
        return fql.linear_fused(fql.linear_fused(x, self.gate_up, activation="swiglu"), self.down, residual=h)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def serve(layer, hidden, prompts, tokens, block_size=64, seed=1, graph=True):
    """(outputs of the prompts, [outputs of each step], (prompt ms, ms a step))."""
    B, gen = len(prompts), torch.Generator(device="cuda").manual_seed(seed)
    blocks = [-(-(n + tokens) // block_size) for n in prompts]  # the blocks every request will need
    cache = fql.KVCache8.empty(sum(blocks), layer.kv_heads, block_size, layer.head_dim)
    table = torch.full((B, max(blocks)), -1, dtype=torch.int32)
    free = list(range(sum(blocks)))
    for b, n in enumerate(blocks):
        for j in range(n):
            table[b, j] = free.pop()
    table = table.cuda()

    def randn(n):
        return torch.randn(n, hidden, generator=gen, device="cuda").to(torch.bfloat16)

    def event():
        e = torch.cuda.Event(enable_timing=True)
        e.record()
        return e

    cu = torch.tensor([0] + prompts).cumsum(0).tolist()
    h, lens, cu = randn(sum(prompts)), i32(prompts), i32(cu)
    begin = event()
    out = layer(h, cache, table, lens, cu, max(prompts))
    times = [(begin, event())]

    h, cu, steps = torch.zeros(B, hidden, dtype=torch.bfloat16, device="cuda"), i32(list(range(B + 1))), []
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # sizes the workspaces; no tokens are appended (lengths 0)
            layer(h, cache, table, torch.zeros_like(lens), cu, 1)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            y = layer(h, cache, table, lens, cu, 1)
    for _ in range(tokens):
        x = randn(B)
        lens += 1
        begin = event()
        if graph:
            h.copy_(x)
            g.replay()
        else:
            y = layer(x, cache, table, lens, cu, 1)
        times.append((begin, event()))
        steps.append(y.clone())
    torch.cuda.synchronize()
    ms = [a.elapsed_time(b) for a, b in times]
    return out, steps, (ms[0], sorted(ms[1:])[len(ms[1:]) // 2] if tokens else None)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--format", default="mxfp8", choices=("fp8", "fp8_block", "mxfp8"))
    p.add_argument("--prompts", default="700,33,1", help="tokens of each request's prompt")
    p.add_argument("--tokens", type=int, default=32, help="single tokens after the prompts")
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", default="32,8,128", help="query heads, kv heads, head dim")
    p.add_argument("--ff", type=int, default=14336)
    a = p.parse_args(argv)
    prompts, (q_heads, kv_heads, head_dim) = ([int(v) for v in s.split(",")] for s in (a.prompts, a.heads))
    layer = DecoderLayer(a.format, a.hidden, q_heads, kv_heads, head_dim, a.ff)
    serve(layer, a.hidden, prompts, 2)  # first launches
    out, steps, (prompt_ms, step_ms) = serve(layer, a.hidden, prompts, a.tokens)
    print(f"{a.format}: prompts of {prompts} tokens {prompt_ms:.3f} ms, a step of {len(prompts)} tokens "
          f"{step_ms * 1e3:.1f} us (HIP graph); rms of the outputs {out.float().square().mean().sqrt():.3f}, "
          f"{torch.stack(steps).float().square().mean().sqrt():.3f}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
