"""One decoder block served from end to end: its W4 linears (bit_gemm_amd.mosaicq)
and what stands between them (bit_gemm_amd.block).

    python examples/decoder_block.py                  # 4096 wide, 32 heads on 8, 16 sequences

    norm -> q,k,v linear -> rotary + cache append -> attention -> o linear -> residual + norm
         -> gate,up linear -> silu(gate) up -> down linear -> residual + norm

Prompts of different lengths are written in one pass, then every sequence decodes one token a step; a step is captured
in a HIP graph once and replayed while the sequences grow. Weights and inputs are random.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_gemm_amd import block as bk  # noqa: E402
from bit_gemm_amd import mosaicq as mq  # noqa: E402


class DecoderBlock:
    """The block's packed linears and norm weights. weights: "q", "k", "v", "o", "gate", "up", "down" [out, in] and
    "norm_attn", "norm_mlp", "norm_next" [hidden], float16 on the GPU."""

    def __init__(self, weights: dict, heads: int, kv_heads: int, head_dim: int, rope: bk.Rope, rho: float = 0.005):
        self.heads, self.kv_heads, self.head_dim, self.rope = heads, kv_heads, head_dim, rope
        pack = {n: mq.mq_pack(weights[n], 128, rho) for n in ("q", "k", "v", "o", "gate", "up", "down")}
        self.qkv = mq.mq_concat([pack[n] for n in ("q", "k", "v")])       # one launch for layers that read the same input
        self.gate_up = mq.mq_concat([pack["gate"], pack["up"]])
        self.o, self.down = pack["o"], pack["down"]
        self.norm_attn, self.norm_mlp, self.norm_next = (weights[n] for n in ("norm_attn", "norm_mlp", "norm_next"))

    def first_norm(self, r):
        """The normed input of the block for a residual stream r [tokens, hidden] (the block before gives both)."""
        return bk.mq_norm_residual(None, r, self.norm_attn)[1]

    def __call__(self, r, h, cache: bk.KVCache, batch: bk.KVBatch, workspace=None):
        """Residual stream r [tokens, hidden] (float32 or float16) and normed input h of a step -> the same of the next
        block."""
        H, K, D = self.heads, self.kv_heads, self.head_dim
        qkv = mq.mq_linear(h, self.qkv).unflatten(1, (H + 2 * K, D))
        q = bk.mq_kv_append(qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:], cache, batch, rope=self.rope)
        a = bk.mq_kv_attention(q, cache, batch, workspace=workspace)
        r, h = bk.mq_norm_residual(mq.mq_linear(a.flatten(1), self.o), r, self.norm_mlp)
        g, u = mq.mq_linear(h, self.gate_up).chunk(2, 1)
        return bk.mq_norm_residual(mq.mq_linear((F.silu(g) * u).contiguous(), self.down), r, self.norm_next)


class Sequences:
    """Block tables and lengths of running sequences over one cache, as a server keeps them."""

    def __init__(self, count: int, longest: int, kv_heads: int, head_dim: int, fmt: str = "int8"):
        width = -(-longest // bk.BLOCK)
        self.cache = bk.KVCache.empty(count * width, count, kv_heads, head_dim, fmt)
        self.table = torch.randperm(count * width, device="cuda").int().view(count, width)
        self.length = torch.zeros(count, dtype=torch.int32, device="cuda")
        self.count, self.longest = count, longest

    def batch(self, new) -> bk.KVBatch:
        """A step that brings new[s] tokens to sequence s; counts them."""
        cu = torch.tensor([0] + list(new), dtype=torch.int32).cumsum(0).int().cuda()
        self.length += cu[1:] - cu[:-1]
        return bk.KVBatch(cu, self.length, self.table, max(new), self.longest)


def random_weights(hidden: int, heads: int, kv_heads: int, head_dim: int, inner: int, seed: int = 0) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes = {"q": (heads * head_dim, hidden), "k": (kv_heads * head_dim, hidden), "v": (kv_heads * head_dim, hidden),
              "o": (hidden, heads * head_dim), "gate": (inner, hidden), "up": (inner, hidden), "down": (hidden, inner)}
    w = {n: (torch.randn(s, generator=g, device="cuda") * s[1] ** -0.5).half() for n, s in shapes.items()}
    return w | {n: (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).half()
                for n in ("norm_attn", "norm_mlp", "norm_next")}


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--sequences", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000, help="longest prompt")
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--format", choices=("int8", "e4m3"), default="int8")
    a = ap.parse_args()
    D = a.hidden // a.heads
    rope = bk.Rope(D, a.prompt + a.steps + 8, theta=500000.0)
    layer = DecoderBlock(random_weights(a.hidden, a.heads, a.kv_heads, D, a.inner), a.heads, a.kv_heads, D, rope)
    seqs = Sequences(a.sequences, a.prompt + a.steps + 8, a.kv_heads, D, a.format)

    new = [max(1, a.prompt - 37 * s) for s in range(a.sequences)]
    batch = seqs.batch(new)
    r = torch.randn((sum(new), a.hidden), device="cuda")
    t = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    h = layer.first_norm(r)
    layer(r, h, seqs.cache, batch)
    t[0].record()
    layer(r, h, seqs.cache, batch)
    t[1].record()

    # a decode step: the same tensors every time, so that a graph can replay it
    one = seqs.batch([1] * a.sequences)
    r = torch.randn((a.sequences, a.hidden), device="cuda")
    h = layer.first_norm(r)
    workspace = torch.empty(max(1, bk.kv_attention_workspace(seqs.cache, one, a.sequences, a.heads)), dtype=torch.uint8,
                            device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(r, h, seqs.cache, one, workspace)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(r, h, seqs.cache, one, workspace)
    t[2].record()
    for _ in range(a.steps):
        seqs.length += 1
        graph.replay()
    t[3].record()
    torch.cuda.synchronize()
    assert all(x.isfinite().all() for x in out)
    print(f"prompts: {sum(new)} tokens in {t[0].elapsed_time(t[1]):.2f} ms; decode: {a.sequences} sequences, "
          f"{t[2].elapsed_time(t[3]) / a.steps * 1e3:.1f} us a step of one block (cache {a.format})")


if __name__ == "__main__":
    main()
