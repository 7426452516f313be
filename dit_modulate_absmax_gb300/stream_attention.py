"""Attention sub-block of a DiT over a video that arrives in chunks.

  python -m dit_modulate_absmax_gb300.stream_attention [--chunks C] [--frames F --height H --width W]
      [--hidden D] [--heads H] [--window N] [--reps R]

Each chunk's tokens go through one block's attention: modulation and NVFP4
packing, the QKV GEMM, rotary positions (time, height, width) of the queries
in place in the GEMM's rows, the keys' rotation and the quantisation of keys
and values into the 8-bit paged cache, attention over everything cached, and
the output projection with its gated residual.  The cache is what remains of
earlier chunks.  The command runs it on synthetic inputs, compares sampled
rows with the definition evaluated in 64 bits on the read-back cache, and
prints the time of each chunk.
"""
from __future__ import annotations

import argparse
import dataclasses

import torch

import dit_modulate_absmax_gb300 as h3
from dit_modulate_absmax_gb300 import build as B
from dit_modulate_absmax_gb300 import workloads as W

HEAD_DIM = 128
AXES = (44, 42, 42)      # channels turned by time, height and width


class StreamAttention:
    """The sub-block with its weights, its cache for one sequence and its buffers."""

    def __init__(self, hidden, heads, max_tokens, page_size=64, window=0, seed=0, device="cuda"):
        self.hidden, self.heads, self.page_size, self.window = hidden, heads, page_size, window
        wide = heads * HEAD_DIM
        base = dataclasses.replace(W.WORKLOADS["qkv"], seed=seed)
        self.qkv_w = self._weight(dataclasses.replace(base, k=hidden, n=3 * wide), device)
        self.out_w = self._weight(dataclasses.replace(base, k=wide, n=hidden, seed=seed + 1), device)
        pages = -(-max_tokens // page_size)
        self.cache = h3.KVCache.empty(pages, page_size, heads, HEAD_DIM, device)
        self.page_table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(device, torch.int32)[None]
        self.freqs = h3.rope_frequencies(AXES, device=device)
        self.held = 0

    @staticmethod
    def _weight(w, device):
        t = W.weights(w, device)
        return t["q"], h3.swizzle_scales(t["sf"][: w.n]), torch.tensor([t["ts"]], dtype=torch.float32, device=device)

    def step(self, x, positions, shift, scale, gate):
        """x [m, hidden] bf16 patterns of a chunk's tokens, positions [m, 3] float32, shift, scale and gate [1, hidden]:
        returns x + gate * attention(...) and appends the chunk to the cache."""
        m, heads = x.shape[0], self.heads
        m_pad, total, dev = -(-m // 16) * 16, self.held + m, x.device
        if total > self.page_table.shape[1] * self.page_size:
            raise ValueError(f"the cache holds {self.page_table.shape[1] * self.page_size} tokens, {total} are wanted")
        ts, packed, sfa = h3.modulate_produce(x, shift, scale, [0, m], m_pad)
        self.qkv = h3.gemm(packed, sfa, ts, *self.qkv_w, m).view(m, 3 * heads, HEAD_DIM)
        q, k, v = self.qkv[:, :heads], self.qkv[:, heads:2 * heads], self.qkv[:, 2 * heads:]
        rope = h3.Rope(positions, self.freqs, AXES)
        h3.rope_axes(q, rope, out=q)
        cu = torch.tensor([0, m], dtype=torch.int32, device=dev)
        held = torch.tensor([self.held], dtype=torch.int32, device=dev)
        h3.kv_cache_write(self.cache, k, v, self.page_table, held, cu, m, rope=rope)
        self.attended, _ = h3.kv_attention(q, self.cache, self.page_table, held + m, cu, m, total, window=self.window)
        self.held = total
        ts, packed, sfa = h3.quantize_pack(self.attended.view(m, heads * HEAD_DIM), m_pad)
        return h3.gemm_gated_residual(packed, sfa, ts, *self.out_w, m, gate, [0, m], x)

    def cached(self):
        """Everything cached as bf16: (keys, values) [held, heads, head_dim], keys turned."""
        cu = torch.tensor([0, self.held], dtype=torch.int32, device=self.page_table.device)
        return h3.kv_cache_read(self.cache, self.page_table, None, cu, self.held, self.held)


def grid_positions(start, frames, height, width, device="cuda"):
    """Time, row and column of each token of ``frames`` frames from frame ``start`` on."""
    t = torch.arange(start, start + frames, dtype=torch.float32)
    axes = torch.meshgrid(t, torch.arange(height, dtype=torch.float32), torch.arange(width, dtype=torch.float32), indexing="ij")
    return torch.stack([a.reshape(-1) for a in axes], 1).contiguous().to(device)


def sampled_error(block, rows):
    """Largest difference of the last chunk's attention from the definition, at some rows, as a fraction of the
    softmax-weighted mean of |v|."""
    keys, values = block.cached()
    m, worst = block.attended.shape[0], 0.0
    for r in rows:
        q = block.qkv[r, : block.heads].view(torch.bfloat16).double()
        lo = max(0, block.held - m + r - block.window + 1) if block.window else 0
        k, v = keys[lo:].double(), values[lo:].double()
        w = torch.softmax(torch.einsum("hd,nhd->hn", q, k) * HEAD_DIM ** -0.5, 1)
        got = block.attended[r].view(torch.bfloat16).double()
        diff = (got - torch.einsum("hn,nhd->hd", w, v)).abs() / torch.einsum("hn,nhd->hd", w, v.abs())
        worst = max(worst, diff.max().item())
    return worst


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--chunks", type=int, default=4)
    ap.add_argument("--frames", type=int, default=3)
    ap.add_argument("--height", type=int, default=30)
    ap.add_argument("--width", type=int, default=52)
    ap.add_argument("--hidden", type=int, default=5376)
    ap.add_argument("--heads", type=int, default=56)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--reps", type=int, default=5, help="timed repetitions of a chunk (the cache is set back)")
    a = ap.parse_args()
    B.build()
    m = a.frames * a.height * a.width
    block = StreamAttention(a.hidden, a.heads, a.chunks * m, window=a.window)
    for c in range(a.chunks):
        w = dataclasses.replace(W.WORKLOADS["qkv"], m=m, k=a.hidden, n=0, seg_off=(0, m), seed=10 + c)
        act = W.activations(w, device="cuda")
        pos = grid_positions(c * a.frames, a.frames, a.height, a.width)
        gate = act["scale"]
        held = block.held
        block.step(act["x"], pos, act["shift"], act["scale"], gate)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(a.reps):
            block.held = held
            block.step(act["x"], pos, act["shift"], act["scale"], gate)
        e1.record()
        err = sampled_error(block, range(0, m, max(1, m // 5)))
        assert h3.h3fp4_device_error() == 0
        print(f"chunk {c}: {m} tokens over {block.held} cached, {e0.elapsed_time(e1) / a.reps:.3f} ms, "
              f"attention off by {err:.1e} of its mean |v|")


if __name__ == "__main__":
    main()
