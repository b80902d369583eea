"""One decode step of an expert decoder layer with 4-bit weights, on random weights.

    h     = x + O( attention( rope( QKV( norm x ) ) ) )        w4a16_gemm, w4a16_rope_append,
                                                               w4a16_paged_attention, w4a16_gemm
    x_new = h + experts( norm h )                              w4a16_moe_layer

Every sequence of the batch gets one new token: its key and value go into the paged cache, it
attends to everything before it, and the layer's output is the next step's input.  Lengths,
positions and slots live on the device, so one captured CUDA graph serves every step.

    python examples/decode_step.py [--batch 8] [--steps 32] [--hidden 2048] ...
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import weight_only_int4_03_gb300 as w4

DEV = "cuda"


class Linear4:
    """A W4A16 weight (u4b8, groups of 128) in the library's tile layout, with its workspace."""

    def __init__(self, g, k, n, max_rows):
        self.k, self.n = k, n
        self.words = torch.randint(-2 ** 31, 2 ** 31 - 1, (k // 8, n), generator=g, device=DEV, dtype=torch.int32)
        self.scales = (torch.rand((k // 128, n), generator=g, device=DEV) * 0.2 + 0.9).div_(5 * k ** 0.5).half()
        self.packed = torch.empty(k * n // 8, dtype=torch.int32, device=DEV)
        w4.w4_repack(self.words, None, self.packed, k, n)
        size = w4.w4a16_workspace_size(max_rows, n, k, 128, w4.W4A16_FLAG_IS_K_FULL)
        self.workspace = torch.zeros(size, dtype=torch.uint8, device=DEV)

    def __call__(self, x, out):
        w4.w4a16_gemm(x, self.packed, out, self.scales, None, None, None, self.workspace, x.shape[0], self.n,
                      self.k, 128, w4.W4A16_TYPE_U4B8, w4.W4A16_FLAG_IS_K_FULL)
        return out


class Experts4:
    """The expert layer's weights: gate and up columns interleaved, then packed expert by expert."""

    def __init__(self, g, hidden, inter, experts, top_k, max_tokens):
        self.hidden, self.inter, self.experts, self.top_k = hidden, inter, experts, top_k
        self.router = (torch.randn((experts, hidden), generator=g, device=DEV) * 2 / hidden ** 0.5).half()
        self.words, self.scales, packed = [], [], []
        for k, n, gated in ((hidden, 2 * inter, True), (inter, hidden, False)):
            words = torch.randint(-2 ** 31, 2 ** 31 - 1, (experts, k // 8, n), generator=g, device=DEV,
                                  dtype=torch.int32)
            scales = (torch.rand((experts, k // 128, n), generator=g, device=DEV) * 0.2 + 0.9).div_(5 * k ** 0.5).half()
            self.words.append(words)
            self.scales.append(scales)
            if gated:
                mixed, mixed_scales = torch.empty_like(words), torch.empty_like(scales)
                w4.w4_gate_up_interleave(words, mixed, experts * k // 8, n)
                w4.w4_gate_up_interleave(scales, mixed_scales, experts * k // 128, n)
                words, scales = mixed, mixed_scales
            tiles = torch.empty((experts, k * n // 8), dtype=torch.int32, device=DEV)
            for e in range(experts):
                w4.w4_repack(words[e], None, tiles[e], k, n)
            packed += [tiles, scales]
        self.packed = packed
        size = w4.w4a16_moe_layer_workspace_size(max_tokens, hidden, inter, experts, top_k)
        self.workspace = torch.zeros(size, dtype=torch.uint8, device=DEV)

    def __call__(self, x, residual, out):
        up, up_s, down, down_s = self.packed
        w4.w4a16_moe_layer(x, self.router, up, up_s, None, down, down_s, None, out, self.workspace, x.shape[0],
                           self.hidden, self.inter, self.experts, self.top_k, 128, w4.W4A16_TYPE_U4B8,
                           w4.W4A16_FLAG_SWIGLU | w4.W4A16_FLAG_MOE_RENORM, residual=residual)
        return out


def rms_norm(x):
    return (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).half()


class DecodeLayer:
    def __init__(self, batch, max_len, hidden=2048, heads=16, kv_heads=4, head_dim=128, inter=1024, experts=16,
                 top_k=4, page=16, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.batch, self.heads, self.kv, self.dim, self.page = batch, heads, kv_heads, head_dim, page
        self.hidden, self.max_len = hidden, max_len
        width = (heads + 2 * kv_heads) * head_dim
        self.qkv = Linear4(g, hidden, width, batch)
        self.o = Linear4(g, heads * head_dim, hidden, batch)
        self.experts = Experts4(g, hidden, inter, experts, top_k, batch)
        freq = 10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64, device=DEV) / head_dim)
        angle = torch.arange(max_len, dtype=torch.float64, device=DEV)[:, None] * freq
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        # Pages are handed out to the sequences in an order of no meaning.
        self.max_pages = (max_len + page - 1) // page
        n_pages = batch * self.max_pages
        self.table = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).view(batch, self.max_pages)
        self.k_cache = torch.zeros((n_pages, page, kv_heads, head_dim), dtype=torch.float16, device=DEV)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=DEV)  # tokens cached so far
        size = w4.w4a16_paged_attention_workspace_size(batch, heads, kv_heads, head_dim)
        self.workspace = torch.zeros(size, dtype=torch.uint8, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        half = dict(dtype=torch.float16, device=DEV)
        self.qkv_out = torch.empty((batch, width), **half)
        self.q = torch.empty((batch, heads * head_dim), **half)
        self.att = torch.empty((batch, heads * head_dim), **half)
        self.proj = torch.empty((batch, hidden), **half)
        self.out = torch.empty((batch, hidden), **half)

    def step(self, x):
        """One new token per sequence: x [batch, hidden] -> the layer's output (a buffer of its own)."""
        b, h, kv, d, page = self.batch, self.heads, self.kv, self.dim, self.page
        positions = self.lens  # the new token's position is the number of those before it
        # Past max_len there is no page to look up: the token is not cached, and the operators report its position
        # and length in their status words.
        at = (positions // page).clamp(max=self.max_pages - 1).long()
        pages = self.table.gather(1, at[:, None]).squeeze(1)
        slots = torch.where(positions < self.max_len, pages.long() * page + (positions % page).long(), -1)
        qkv = self.qkv(rms_norm(x), self.qkv_out)
        width = qkv.shape[1]
        w4.w4a16_rope_append(qkv, qkv[:, h * d:], qkv[:, (h + kv) * d:], self.q, self.k_cache, self.v_cache,
                             self.cos_sin, positions, slots, self.status, b, h, kv, d, d, [d // 2],
                             self.max_len, page, self.k_cache.shape[0], ldq=width, ldk=width, ldv=width)
        self.lens += 1
        w4.w4a16_paged_attention(self.q, self.k_cache, self.v_cache, self.att, self.table, self.lens,
                                 self.workspace, b, h, kv, d, page, self.k_cache.shape[0], self.max_pages, d ** -0.5)
        mid = x + self.o(self.att, self.proj)
        return self.experts(rms_norm(mid), mid, self.out)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=4)
    args = ap.parse_args(argv)
    layer = DecodeLayer(args.batch, args.steps + 16, hidden=args.hidden, inter=args.inter, experts=args.experts,
                        top_k=args.top_k)
    x = torch.randn((args.batch, args.hidden), dtype=torch.float16, device=DEV)
    for _ in range(3):  # warm up outside the graph
        layer.step(x)
    layer.lens.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(rms_norm(layer.step(x)))  # stands in for the next tokens
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    bits = int(layer.status.item()) | w4.w4a16_status(layer.workspace)
    print(f"{args.steps} steps of {args.batch} sequences: {start.elapsed_time(end) / args.steps * 1e3:.1f} us a step, "
          f"lengths now {layer.lens.tolist()}, device status {bits}, |x| {float(x.float().abs().mean()):.3f}")


if __name__ == "__main__":
    main()
