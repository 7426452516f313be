"""The attention path's operators as they are used together: a block whose
queries and keys are normed, over a video with a window and a first frame that
stays; a serving step whose tables are made on the GPU, captured and replayed."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_cache import _dev, _patterns
from test_gpu_kv_sinks import check_rows

pytestmark = pytest.mark.gpu


def _values(t):
    return O.bf16_values(_patterns(t))


def _cached(c, table, length):
    return [O.gather(O.cache_values(t.cpu().numpy(), s.cpu().numpy()), table, length)
            for t, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))]


@pytest.mark.parametrize("chunks,window,sinks", [([(2, 5, 7), (1, 3, 11), (1, 1, 1), (3, 6, 9)], 60, 35),
                                                 ([(1, 4, 30), (2, 1, 1), (1, 10, 13)], 0, 0)])
def test_block_with_norms_over_a_video(h3, chunks, window, sinks):
    from dit_modulate_absmax_gb300 import stream_attention as S
    heads = 2
    block = S.StreamAttention(256, heads, sum(f * r * c for f, r, c in chunks), page_size=32, window=window, seed=3, sinks=sinks,
                              qk_norm=True)
    gen, frame = torch.Generator().manual_seed(1), 0
    freqs = block.freqs.cpu().numpy()
    for f, r, c in chunks:
        m = f * r * c
        x = torch.randn(m, 256, generator=gen).bfloat16().view(torch.int16).cuda()
        shift, scale, gate = [(torch.randn(1, 256, generator=gen) * 0.2).bfloat16().view(torch.int16).cuda() for _ in range(3)]
        pos = S.grid_positions(frame, f, r, c)
        out = block.step(x, pos, shift, scale, gate)
        frame += f
        pad = -(-m // 16) * 16                                # the projection by hand, before its rows are normed
        ts, packed, sfa = h3.modulate_produce(x, shift, scale, [0, m], pad)
        raw = _values(h3.gemm(packed, sfa, ts, *block.qkv_w, m).view(m, 3 * heads, 128))

        def turn(z):
            return O.rope(z, pos.cpu().numpy(), freqs, S.AXES, "interleaved")

        for at, w in ((0, block.norms[0]), (heads, block.norms[1])):
            ref, mag = O.norm_rope(raw[:, at:at + heads], w.double().cpu().numpy(), 1e-6, turn)
            got = _values(block.qkv[:, at:at + heads])
            assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + 2.0 ** -19 * mag + 1e-38).all()
        table = block.page_table[0].cpu().numpy()
        k, v = _cached(block.cache, table, block.held)
        q = _values(block.qkv[:, :heads])
        ref, _, A, P, T = O.attention(q, k, v, 128 ** -0.5, window=window, sinks=sinks)
        e = 2.0 ** -17 * P
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 4 * e[..., None]) * A + block.held * 2.0 ** -22 * T[..., None] + 1e-38
        assert (np.abs(_values(block.attended) - ref) <= tol).all()
        ts, packed, sfa = h3.quantize_pack(block.attended.view(m, heads * 128), pad)
        assert torch.equal(out, h3.gemm_gated_residual(packed, sfa, ts, *block.out_w, m, gate, [0, m], x))
        assert S.sampled_error(block, range(0, m, max(1, m // 3))) < 0.05
    assert h3.h3fp4_device_error() == 0


class _Server:
    """Requests behind a shared prompt: each step makes the tables of its new tokens, norms and turns queries and keys, writes
    the cache and attends, all from lengths that lie on the device."""

    def __init__(self, h3, batch, most_new, prompt, seed, page=32, heads=8, kv_heads=2, dim=64):
        self.h3, self.batch, self.most, self.page = h3, batch, most_new, page
        self.prompt, self.heads, self.kv_heads, self.dim = prompt, heads, kv_heads, dim
        self.room = 12
        pages = batch * self.room + -(-prompt // page) + 3
        self.cache = h3.KVCache.empty(pages, page, kv_heads, dim)
        for codes in (self.cache.k_codes, self.cache.v_codes):
            codes.zero_()                                     # (two servers' caches are compared as a whole)
        free = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int().cuda()
        used = -(-prompt // page)
        self.prefix_table, self.free = free[None, :used].contiguous(), free[used:].contiguous()
        g = torch.Generator().manual_seed(seed + 1)
        pk = torch.randn(prompt, 2 * kv_heads, dim, generator=g).bfloat16().cuda()
        h3.kv_cache_write(self.cache, pk[:, :kv_heads], pk[:, kv_heads:], self.prefix_table, _dev([0]), _dev([0, prompt]), prompt)
        self.rows = batch * most_new
        self.table = torch.full((batch, self.room), -1, dtype=torch.int32, device="cuda")
        self.held, self.count, self.at = _dev([0] * batch), _dev([1] * batch), _dev([0])
        self.qkv = torch.zeros(self.rows, heads + 2 * kv_heads, dim, dtype=torch.bfloat16, device="cuda")
        self.w = [(1 + 0.2 * torch.randn(dim, generator=g)).cuda() for _ in "qk"]
        self.freqs = h3.rope_frequencies((dim,))
        self.p_len = _dev([prompt])

    def step(self):
        h3, hq, hk = self.h3, self.heads, self.kv_heads
        t = h3.kv_tables(self.held, self.count, self.table, self.free, self.at, self.page, self.cache.num_pages, self.rows, self.most)
        rope = h3.Rope(t.positions[:, None], self.freqs, (self.dim,), layout="halves")
        q, k = h3.norm_rope(self.qkv[:, :hq], self.qkv[:, hq:hq + hk], q_weight=self.w[0], k_weight=self.w[1], rope=rope)
        h3.kv_cache_write(self.cache, k, self.qkv[:, hq + hk:], self.table, self.held, t.cu_tokens, self.most)
        ends = torch.stack([t.cu_tokens[0], t.cu_tokens[-1]])
        prefix = h3.SharedPrefix(self.prefix_table, self.p_len, ends, self.rows, self.prompt)
        most = self.room * self.page
        shared = h3.kv_attention_shared(q, self.cache, prefix, self.table, t.kv_len, t.cu_tokens, self.most, most, causal=True,
                                        return_lse=True)
        near = h3.kv_attention(q, self.cache, self.table, t.kv_len, t.cu_tokens, self.most, most, causal=True, window=40, sinks=5,
                               return_lse=True)
        return t, q, k, shared, near

    def advance(self, t):
        self.held.copy_(t.kv_len)
        self.at.copy_(t.free_at)


@pytest.mark.parametrize("batch,most", [(3, 1), (40, 1), (5, 37)])
def test_serving_steps_captured_and_by_hand(h3, batch, most):
    """Steps of changing lengths: from one captured graph, to the bits of the calls made one by one, whose last results meet
    the definitions on what the cache holds."""
    eager, replayed = [_Server(h3, batch, most, 150, 7) for _ in range(2)]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        out = replayed.step()
    g = torch.Generator().manual_seed(batch)
    for i in range(6):
        count = torch.randint(0 if i else 1, most + 1, (batch,), generator=g).int().cuda()
        x = torch.randn(eager.qkv.shape, generator=g).mul(1.5).bfloat16().cuda()
        for server in (eager, replayed):
            server.count.copy_(count)
            server.qkv.copy_(x)
        t, q, k, shared, near = eager.step()
        graph.replay()
        torch.cuda.synchronize()
        n = int(t.cu_tokens[-1])
        for a, b in zip(t, out[0]):
            assert torch.equal(a, b)
        for a, b in ((q, out[1]), (k, out[2]), (shared[0], out[3][0]), (shared[1], out[3][1]), (near[0], out[4][0]), (near[1], out[4][1])):
            assert torch.equal(a[:n], b[:n])
        assert torch.equal(eager.table, replayed.table) and torch.equal(eager.cache.k_codes, replayed.cache.k_codes)
        held, cu, lens = eager.held.tolist(), t.cu_tokens.tolist(), t.kv_len.tolist()
        table, prefix = eager.table.cpu().numpy(), eager.prefix_table[0].cpu().numpy()
        pk, pv = _cached(eager.cache, prefix, 150)
        qv = _values(q)
        for b in range(batch):
            at = slice(cu[b], cu[b + 1])
            if at.start == at.stop:
                continue
            slots = [int(table[b, p // 32]) * 32 + p % 32 for p in range(held[b], lens[b])]
            assert t.slots[at].tolist() == slots and t.positions[at].tolist() == [float(p) for p in range(held[b], lens[b])]
            kk, vv = _cached(eager.cache, table[b], lens[b])
            check_rows(qv[at], np.concatenate([pk, kk]), np.concatenate([pv, vv]), _values(shared[0])[at], shared[1][at].cpu().numpy(),
                       64 ** -0.5, 150 + lens[b], causal=True, before=150)
            check_rows(qv[at], kk, vv, _values(near[0])[at], near[1][at].cpu().numpy(), 64 ** -0.5, lens[b], causal=True, window=40, sinks=5)
        for server, tables in ((eager, t), (replayed, out[0])):
            server.advance(tables)
    assert h3.h3fp4_device_error() == 0
