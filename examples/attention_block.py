"""One attention block served from an 8-bit paged cache: 4-bit QKV projection, rotary
positions and cache append, attention, FP8 output projection.

A prompt goes through in chunks, then single tokens in a CUDA graph, all on one stream:
each call is queued behind the one that feeds it, and nothing is allocated or read back
between them. Prints the time of a decode step and how far the outputs are from the same
block in FP32 with an unquantised cache.

    python examples/attention_block.py [--batch B] [--prompt P] [--steps S]
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import fp8_weight_only_gemm_gb300 as w8  # noqa: E402


class AttentionBlock:
    """Weights, cache and page table of one block; every sequence has the same length."""

    def __init__(self, batch, max_len, hidden=2048, heads=16, kv_heads=2, head_dim=128, page_size=64, group=128, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.batch, self.heads, self.kv_heads, self.head_dim = batch, heads, kv_heads, head_dim
        n = (heads + 2 * kv_heads) * head_dim
        # 4-bit codes with a scale and a zero point for each group, as a 4-bit checkpoint holds them
        self.w_qkv = torch.randint(0, 256, (n, hidden // 2), generator=g, dtype=torch.uint8, device="cuda")
        self.s_qkv = torch.rand(n, hidden // group, generator=g, device="cuda") * 0.4 / hidden ** 0.5
        self.z_qkv = torch.randint(6, 10, (n, hidden // group), generator=g, dtype=torch.uint8, device="cuda")
        w_out = torch.randn(hidden, heads * head_dim, generator=g, device="cuda") / (heads * head_dim) ** 0.5
        self.w_out, self.s_out = w8.quantize_weights(w_out)
        pages = -(-max_len // page_size)
        self.cache = w8.KVCache.empty(batch * pages, page_size, kv_heads, head_dim)
        self.table = torch.randperm(batch * pages, generator=g, device="cuda").to(torch.int32).view(batch, pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float32) / head_dim)
        angle = torch.arange(max_len, device="cuda", dtype=torch.float32)[:, None] * inv
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()
        self.workspaces = {}

    def workspace(self, tokens):
        """Of a call with this many tokens a sequence; made once, before any capture."""
        if tokens not in self.workspaces:
            n = w8.kv_attention_workspace_bytes(self.cache, self.batch, tokens, self.heads)
            self.workspaces[tokens] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return self.workspaces[tokens]

    def forward(self, x):
        """x: bf16 [batch * tokens, hidden], the next tokens of every sequence."""
        tokens = x.shape[0] // self.batch
        self.lens += tokens
        qkv = w8.gemm_w4(x, self.w_qkv, self.s_qkv, zeros=self.z_qkv).view(x.shape[0], -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        w8.kv_append(self.cache, k, v, self.table, self.lens, self.cos, self.sin, q=q, q_out=q)   # rotated in place
        o = w8.kv_attention(self.cache, q, self.table, self.lens, workspace=self.workspace(tokens))
        return w8.gemm(o.view(x.shape[0], -1), self.w_out, self.s_out)

    def plain(self, x):
        """The whole of x, [batch, length, hidden], in FP32 with an unquantised cache."""
        w = torch.stack((self.w_qkv & 15, self.w_qkv >> 4), -1).flatten(1).float()
        group = w.shape[1] // self.s_qkv.shape[1]
        w = (w - self.z_qkv.repeat_interleave(group, 1)) * self.s_qkv.repeat_interleave(group, 1)
        length, r = x.shape[1], self.head_dim // 2
        qkv = (x.float() @ w.T).view(self.batch, length, -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 2)
        cos, sin = self.cos[:length, None], self.sin[:length, None]
        q, k = (torch.cat((t[..., :r] * cos - t[..., r:] * sin, t[..., r:] * cos + t[..., :r] * sin), -1) for t in (q, k))
        k, v = (t.repeat_interleave(self.heads // self.kv_heads, 2) for t in (k, v))
        s = torch.einsum("bihd,bjhd->bhij", q, k) * self.head_dim ** -0.5
        s.masked_fill_(torch.ones(length, length, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v).flatten(2)
        rows = torch.arange(self.w_out.shape[0], device="cuda")[:, None] // 128
        cols = torch.arange(self.w_out.shape[1], device="cuda")[None] // 128
        return o @ (self.w_out.view(torch.float8_e4m3fn).float() * self.s_out[rows, cols]).T


def run(batch=4, prompt=500, chunk=192, steps=64, **config):
    """Outputs [batch, prompt + steps, hidden], the same from the plain form, and the us of a step."""
    length = prompt + steps
    block = AttentionBlock(batch, length, **config)
    hidden = block.w_out.shape[0]
    x = torch.randn(batch, length, hidden, device="cuda").to(torch.bfloat16)
    outs = []
    for at in range(0, prompt, chunk):
        part = x[:, at:min(at + chunk, prompt)]
        outs.append(block.forward(part.reshape(-1, hidden)).view(batch, -1, hidden))

    x_step = torch.zeros(batch, hidden, dtype=torch.bfloat16, device="cuda")
    block.workspace(1)
    lens = block.lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):          # a first call outside the capture; its token is written again below
        block.forward(x_step)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y_step = block.forward(x_step)
    block.lens.copy_(lens)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for i in range(steps):
        x_step.copy_(x[:, prompt + i])
        graph.replay()
        outs.append(y_step.clone()[:, None])
    end.record()
    torch.cuda.synchronize()
    code, where, _ = w8.device_status()
    if code:
        raise RuntimeError(f"device status {code} at {where}")
    return torch.cat(outs, 1), block.plain(x), begin.elapsed_time(end) / steps * 1e3


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=500)
    p.add_argument("--steps", type=int, default=64)
    a = p.parse_args()
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    got, want, us = run(a.batch, a.prompt, steps=a.steps)
    err = (got.float() - want).norm() / want.norm()
    print(f"{a.batch} sequences of {a.prompt} + {a.steps} tokens: {us:.1f} us a step, relative error {err:.4f} (8-bit cache against FP32)")


if __name__ == "__main__":
    main()
