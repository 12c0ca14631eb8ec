"""An attention layer over the 8-bit paged key/value cache: prompts, then single tokens.

    x -> W8A16 projection to q, k, v     wq_linear
      -> rotary positions on q and k     wq_rope          (one call, in place on the fused rows)
      -> k, v into the cache, 8 bits     wq_kv_write
      -> attention over the cache        wq_kv_attention
      -> W4A16 output projection + x     wq_linear_residual

A few prompts of different lengths go through the layer in one ragged batch; then every
sequence takes one token a step, the whole step captured in a HIP graph that is replayed
while the positions advance on the device.  Random weights, no files.

    python examples/attention_layer.py [--prompts 700,33,1900] [--steps 32]
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import gemm_decode_amd.wq as wq


class AttentionLayer:
    """Weights, rotary table and cache of one layer.  w_qkv: fp32 [(heads + 2 kv_heads) * head_dim]
    [hidden], w_out: fp32 [hidden][heads * head_dim]; every sequence has room for `room` tokens."""

    def __init__(self, w_qkv, w_out, heads, kv_heads, head_dim, seqs, room, page_tokens=64):
        self.heads, self.kv_heads, self.head_dim, self.room = heads, kv_heads, head_dim, room
        device = w_qkv.device
        self.w_qkv, self.w_out = wq.quantize(w_qkv, "w8pc"), wq.quantize(w_out, "w4g128")
        self.inv_freq = 10000.0 ** (-torch.arange(head_dim // 2, device=device, dtype=torch.float32) * 2 / head_dim)
        width = -(-room // page_tokens)
        self.cache = wq.KVCache(seqs * width, page_tokens, kv_heads, head_dim, device=device)
        order = torch.randperm(seqs * width, device=device)   # pages come in any order
        self.table = order.to(torch.int32).view(seqs, width).contiguous()

    def plan(self, batch, tokens):
        """Buffers of a step of this many token rows, kept from step to step."""
        dev, D = self.table.device, self.head_dim
        buf = lambda n: torch.empty(tokens, n, dtype=torch.bfloat16, device=dev)
        bytes_ = [wq.wq_workspace_size(self.w_qkv, tokens), wq.wq_workspace_size(self.w_out, tokens),
                  wq.wq_kv_attention_workspace_size(self.cache, batch, self.heads, tokens, self.room)]
        return {"qkv": buf((self.heads + 2 * self.kv_heads) * D), "o": buf(self.heads * D),
                "ws": wq.workspace(max(bytes_), device=dev)}

    def forward(self, x, y, batch, positions, plan):
        """y = x + layer(x): x, y bf16 [tokens][hidden], positions int32 [tokens]; allocates nothing."""
        H, KV, D, T = self.heads, self.kv_heads, self.head_dim, x.shape[0]
        wq.wq_linear(self.w_qkv, x, plan["qkv"], ws=plan["ws"])
        rows = plan["qkv"].view(T, H + 2 * KV, D)
        q, k, v = rows[:, :H], rows[:, H:H + KV], rows[:, H + KV:]
        wq.wq_rope(rows[:, :H + KV], rows[:, :H + KV], positions, self.inv_freq)
        wq.wq_kv_write(self.cache, batch, k, v)
        wq.wq_kv_attention(self.cache, batch, q, plan["o"].view(T, H, D), D ** -0.5, max_kv=self.room, ws=plan["ws"])
        wq.wq_linear_residual(self.w_out, plan["o"], x, y, ws=plan["ws"])


def prompt_batch(layer, counts):
    """Ragged prompts that all start at position 0."""
    dev = layer.table.device
    offsets = torch.tensor([0] + list(counts), dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
    positions = torch.cat([torch.arange(n, dtype=torch.int32, device=dev) for n in counts])
    starts = torch.zeros(len(counts), dtype=torch.int32, device=dev)
    return wq.KVBatch(layer.table, starts, offsets, max_tokens=max(counts)), positions


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompts", default="700,33,1900")
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    counts = [int(n) for n in a.prompts.split(",")]
    hidden, seqs = 2048, len(counts)
    torch.manual_seed(0)
    heads, kv_heads, D = 16, 4, 128
    rnd = lambda n, k: torch.randn(n, k, device="cuda") * k ** -0.5
    layer = AttentionLayer(rnd((heads + 2 * kv_heads) * D, hidden), rnd(hidden, heads * D), heads, kv_heads, D, seqs,
                           room=max(counts) + a.steps)

    tokens = sum(counts)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    y = torch.empty_like(x)
    batch, positions = prompt_batch(layer, counts)
    layer.forward(x, y, batch, positions, layer.plan(batch, tokens))
    print(f"{seqs} prompts, {tokens} tokens: |y - x| = {(y.float() - x.float()).abs().mean().item():.4f}")

    # a token per sequence and step: position and start are the same tensor
    starts = torch.tensor(counts, dtype=torch.int32, device="cuda")
    batch = wq.KVBatch(layer.table, starts)
    x1 = torch.randn(seqs, hidden, device="cuda").bfloat16()
    y1 = torch.empty_like(x1)
    plan = layer.plan(batch, seqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x1, y1, batch, starts, plan)      # (writes the tokens that the first replay writes again)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x1, y1, batch, starts, plan)
    e0, e1 = torch.cuda.Event(True), torch.cuda.Event(True)
    e0.record()
    for _ in range(a.steps):
        graph.replay()
        starts.add_(1)      # (a model would put the next token's row into x1 here)
    e1.record()
    torch.cuda.synchronize()
    assert torch.isfinite(y1).all()
    kv16 = 2 * 2 * sum(counts) * layer.kv_heads * layer.head_dim
    print(f"{a.steps} steps of {seqs} tokens: {e0.elapsed_time(e1) / a.steps * 1e3:.1f} us a step; the cache "
          f"holds {kv16 / 2 ** 20:.1f} MiB of 16-bit keys and values in half of that")


if __name__ == "__main__":
    main()
