"""The attention sub-block over a video in chunks: its cache and attention
against the 64-bit forms of what its own GEMM produced, and its output
against the block's calls made one by one."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_cache import _patterns

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunks,window", [([(2, 5, 7), (1, 3, 11), (1, 1, 1), (3, 6, 9)], 0), ([(1, 4, 30), (2, 1, 1), (1, 10, 13)], 50)])
def test_chunks_against_64_bits(h3, chunks, window):
    from dit_modulate_absmax_gb300 import stream_attention as S
    hidden, heads = 256, 2
    most = sum(f * r * c for f, r, c in chunks)
    block = S.StreamAttention(hidden, heads, most, page_size=32, window=window, seed=3)
    gen = torch.Generator().manual_seed(1)
    freqs = block.freqs.cpu().numpy()
    ref_k = np.zeros((0, heads, 128))
    mag_k = np.zeros((0, heads, 128))
    ref_v = np.zeros((0, heads, 128))
    frame = 0
    for f, r, c in chunks:
        m = f * r * c
        x = torch.randn(m, hidden, generator=gen).bfloat16().view(torch.int16).cuda()
        shift, scale, gate = [(torch.randn(1, hidden, generator=gen) * 0.2).bfloat16().view(torch.int16).cuda() for _ in range(3)]
        pos = S.grid_positions(frame, f, r, c)
        held = block.held
        out = block.step(x, pos, shift, scale, gate)
        frame += f
        # the same calls by hand
        pad = -(-m // 16) * 16
        ts, packed, sfa = h3.modulate_produce(x, shift, scale, [0, m], pad)
        qkv = h3.gemm(packed, sfa, ts, *block.qkv_w, m).view(m, 3 * heads, 128)
        assert torch.equal(qkv[:, heads:], block.qkv[:, heads:])
        raw = O.bf16_values(_patterns(qkv))
        q, mag = O.rope(raw[:, :heads], pos.cpu().numpy(), freqs, S.AXES, "interleaved")
        got_q = O.bf16_values(_patterns(block.qkv[:, :heads]))
        assert (np.abs(got_q - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -20 * mag).all()
        k, mag = O.rope(raw[:, heads:2 * heads], pos.cpu().numpy(), freqs, S.AXES, "interleaved")
        ref_k, mag_k, ref_v = np.concatenate([ref_k, k]), np.concatenate([mag_k, mag]), np.concatenate([ref_v, raw[:, 2 * heads:]])
        # cached: a rounding to bf16 (keys), then one to E4M3 (2^-4, or half its smallest step, 2^-10, times the largest
        # scale, for each time a page's scale grew and once at first)
        keys, values = [O.bf16_values(_patterns(t)) for t in block.cached()]
        ks, vs = block.cache.k_scale.max().item(), block.cache.v_scale.max().item()
        times = len(chunks)
        assert (np.abs(keys - ref_k) <= times * (2.0 ** -4 * 1.07 * np.abs(ref_k) + 2.0 ** -10 * ks) + 2.0 ** -8 * mag_k).all()
        assert (np.abs(values - ref_v) <= times * (2.0 ** -4 * 1.07 * np.abs(ref_v) + 2.0 ** -10 * vs)).all()
        # attention: of the rows' own queries over what the cache holds
        ref, _, A, P, T = O.attention(got_q, keys, values, 128 ** -0.5, False, window)
        att = O.bf16_values(_patterns(block.attended))
        e = 2.0 ** -17 * P
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 4 * e[..., None]) * A + block.held * 2.0 ** -22 * T[..., None] + 1e-38
        assert (np.abs(att - ref) <= tol).all()
        assert S.sampled_error(block, range(0, m, 7)) < 0.01
        # output projection
        ts, packed, sfa = h3.quantize_pack(block.attended.view(m, heads * 128), pad)
        want = h3.gemm_gated_residual(packed, sfa, ts, *block.out_w, m, gate, [0, m], x)
        assert torch.equal(out, want)
        assert block.held == held + m
    with pytest.raises(ValueError, match="holds"):
        block.page_table = block.page_table[:, :1].contiguous()
        block.step(x, pos, shift, scale, gate)
    assert h3.h3fp4_device_error() == 0
