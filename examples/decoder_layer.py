"""One decoder layer, decoding a batch of sequences token by token with the
library's calls alone: norm into the 8-bit operand, QKV product, rotation with
the append to the paged cache, attention, quantisation, output product, norm,
router and int4 expert stage. Random weights, one CUDA graph per step.

    python examples/decoder_layer.py [--batch 8] [--steps 64]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import awq_int4_moe_gb300 as awq  # noqa: E402

BLOCK = awq.FP8_BLOCK
EPS = 1e-6


def fp8_weight(w):
    """A weight [N][K] as e4m3 and a scale per 128 x 128 block, for fp8_gemm."""
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    wide = torch.zeros(nb * BLOCK, kb * BLOCK, device=w.device)
    wide[:n, :k] = w
    blocks = wide.view(nb, BLOCK, kb, BLOCK)
    scales = blocks.abs().amax((1, 3)).clamp(min=1e-12) / 448
    q = (blocks / scales[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * BLOCK, kb * BLOCK)
    return q[:n, :k].contiguous(), scales.contiguous()


class DecoderLayer:
    """Weights, cache and buffers of one layer for `batch` sequences of up to
    `max_len` tokens. step() decodes one token of each."""

    def __init__(self, batch: int, max_len: int, seed: int = 0, q_heads: int = 20, kv_heads: int = 4, dim: int = 128,
                 page: int = 16, rotary_base: float = 10000.0):
        import synth
        import synth.device as sd
        dev, half, f8 = "cuda", torch.float16, torch.float8_e4m3fn
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        expert = synth.ExpertShape(num_experts=512, top_k=10, hidden=2560, inter=160, meta_bytes=4)
        self.shape = awq.Shape.of(expert)
        hidden, E, I = expert.hidden, expert.num_experts, expert.inter
        self.batch, self.q_heads, self.kv_heads, self.dim = batch, q_heads, kv_heads, dim
        qkv_cols = (q_heads + 2 * kv_heads) * dim

        def normal(*shape, std=1.0):
            return torch.randn(shape, generator=g, device=dev) * std

        self.norm1, self.norm2 = ((1 + normal(hidden, std=0.1)).to(half) for _ in range(2))
        self.qkv_w, self.qkv_s = fp8_weight(normal(qkv_cols, hidden, std=hidden ** -0.5))
        self.o_w, self.o_s = fp8_weight(normal(hidden, q_heads * dim, std=(q_heads * dim) ** -0.5))
        self.router = normal(E, hidden, std=hidden ** -0.5)
        # the expert stage's banks, prepared once
        canon = [torch.empty((E, hidden // 8, 2 * I), dtype=torch.int32, device=dev),
                 torch.empty((E, hidden // 32, 2 * I, 4), dtype=torch.uint8, device=dev),
                 torch.empty((E, I // 8, hidden), dtype=torch.int32, device=dev),
                 torch.empty((E, I // 32, hidden, 4), dtype=torch.uint8, device=dev)]
        sd.fill_layer(expert, seed, 0, *canon)
        self.banks = [torch.empty_like(t) for t in canon]
        self.experts = awq.moe_prepare_weights(self.shape, awq.Weights.of(*canon), awq.Weights.of(*self.banks))
        torch.cuda.synchronize()

        angle = torch.arange(max_len, device=dev, dtype=torch.float64)[:, None] * \
            rotary_base ** (-torch.arange(0, dim, 2, device=dev, dtype=torch.float64) / dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        pages = -(-max_len // page)
        self.page = page
        self.k_cache = torch.zeros((batch * pages, page, kv_heads, dim), dtype=half, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        order = torch.randperm(batch * pages, generator=g, device=dev)
        self.page_table = order.view(batch, pages).int()
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.rows = torch.arange(batch, device=dev)

        # a step's buffers
        self.x = torch.zeros((batch, hidden), dtype=half, device=dev)            # in: the token's embedding; out: the experts' sum
        self.residual = torch.zeros_like(self.x)
        self.h = torch.empty_like(self.x)
        self.h_q = torch.empty((batch, hidden), dtype=f8, device=dev)
        self.h_s = torch.empty((batch, -(-hidden // BLOCK)), device=dev)
        self.qkv = torch.empty((batch, qkv_cols), dtype=half, device=dev)
        self.attn = torch.empty((batch, q_heads, dim), dtype=half, device=dev)
        self.attn_q = torch.empty((batch, q_heads * dim), dtype=f8, device=dev)
        self.attn_s = torch.empty((batch, -(-q_heads * dim // BLOCK)), device=dev)
        self.o = torch.empty_like(self.x)
        self.ids = torch.empty((batch, expert.top_k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((batch, expert.top_k), device=dev)
        self.attn_ws = torch.zeros(awq.paged_attention_workspace_bytes(dim), dtype=torch.uint8, device=dev)
        self.moe_ws_bytes = awq.moe_workspace_bytes(self.shape, batch)
        self.moe_ws = torch.zeros(self.moe_ws_bytes, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def attention_half(self):
        """x -> o: norm, QKV, rotation and append, attention, output product."""
        b, qh, kh, d = self.batch, self.q_heads, self.kv_heads, self.dim
        awq.add_rmsnorm(self.x, self.norm1, EPS, residual=self.residual, residual_out=self.residual, out_q=self.h_q,
                        out_scales=self.h_s)
        awq.fp8_gemm(self.h_q, self.h_s, self.qkv_w, self.qkv_s, self.qkv, self.status)
        heads = self.qkv.view(b, qh + 2 * kh, d)
        q, k, v = heads[:, :qh], heads[:, qh:qh + kh], heads[:, qh + kh:]
        positions = self.seq_lens.clone()                # the new token's, then the length with it
        at = positions.long()
        slots = self.page_table[self.rows, at // self.page].long() * self.page + at % self.page
        self.seq_lens += 1
        awq.rope_append(q, k, v, positions, self.cos_sin, slots, self.k_cache, self.v_cache, self.status)
        awq.paged_attention(q, self.k_cache, self.v_cache, self.page_table, self.seq_lens, self.attn, self.attn_ws, self.status)
        awq.quantize_fp8(self.attn.view(b, qh * d), self.attn_q, self.attn_s)
        awq.fp8_gemm(self.attn_q, self.attn_s, self.o_w, self.o_s, self.o, self.status)

    def expert_half(self):
        """o -> x: norm, router, expert stage."""
        awq.add_rmsnorm(self.o, self.norm2, EPS, residual=self.residual, residual_out=self.residual, out=self.h)
        logits = self.h.float() @ self.router.t()
        awq.moe_layer_logits(self.h, logits, self.batch, self.shape, self.experts, self.x, self.ids, self.weights, self.moe_ws,
                             self.moe_ws_bytes, self.status)

    def step(self):
        self.attention_half()
        self.expert_half()


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--steps", type=int, default=64)
    a = p.parse_args()
    layer = DecoderLayer(a.batch, a.steps + 8)
    layer.x.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())        # weights, zeroed workspaces and x were made there
    with torch.cuda.stream(side):
        for _ in range(2):                               # set-up outside the graph
            layer.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if int(layer.status):
        raise SystemExit(f"device status {int(layer.status)}: {awq.status_string(int(layer.status))}")
    print(f"batch {a.batch}: {a.steps} steps, {start.elapsed_time(end) / a.steps * 1000:.1f} us each, "
          f"lengths {layer.seq_lens.tolist()}, output norm {layer.x.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
