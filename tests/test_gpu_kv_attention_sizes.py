"""Attention over the 8-bit paged cache where its work is divided: the last
sizes of a variant and the first of the next, many sequences, segments of
many pages, codes past 32 bits.  Bounds as in test_gpu_kv_attention."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_attention import _check, _filled, _run
from test_gpu_kv_cache import _dev, _tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,group", [(8, 1), (9, 1), (16, 1), (17, 1), (3, 8), (31, 1), (4, 8), (33, 1), (17, 2), (5, 7)])
@pytest.mark.parametrize("lengths", [(40, 129), (1_500, 900)])
def test_numbers_of_rows(h3, new, group, lengths):
    rng = np.random.default_rng(new)
    table, pages = _tables(rng, lengths, 32)
    c = _filled(h3, rng, table, lengths, pages, 2, 32, 64)
    cu = [0, new, 2 * new]
    q = torch.randn(2 * new, 2 * group, 64, generator=torch.Generator().manual_seed(new)).mul(2).bfloat16().cuda()
    for causal, window in ((True, 0), (True, 37), (False, 0)):
        out, lse = _run(h3, q, c, table, lengths, cu, new, causal=causal, window=window)
        _check(h3, q, c, table, lengths, cu, out, lse, causal=causal, window=window)
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("most", [1, 2, 40])
def test_many_sequences_of_all_lengths(h3, most):
    """More sequences than a CTA has threads, empty ones and ones without queries among them."""
    rng = np.random.default_rng(most)
    lengths = [int(n) for n in rng.integers(0, 400, 300)]
    lengths[7] = lengths[299] = 0
    lengths[150] = 1_400
    new = [int(n) for n in rng.integers(0, most + 1, 300)]
    new[0] = most
    table, pages = _tables(rng, lengths, 16)
    c = _filled(h3, rng, table, lengths, pages, 1, 16, 64)
    cu = np.cumsum([0] + new)
    q = torch.randn(int(cu[-1]), 2, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    for window in (0, 30):
        out, lse = _run(h3, q, c, table, lengths, cu, most, causal=True, window=window)
        _check(h3, q, c, table, lengths, cu, out, lse, causal=True, window=window)
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("most_kv", [900, 1 << 20])
def test_largest_length_is_only_a_bound(h3, new, most_kv):
    """A larger max_kv changes how the work is spread, not what comes out."""
    rng = np.random.default_rng(2)
    lengths = [900, 33]
    table, pages = _tables(rng, lengths, 64)
    c = _filled(h3, rng, table, lengths, pages, 2, 64, 128)
    cu = [0, new, 2 * new]
    q = torch.randn(2 * new, 16, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    out, lse = h3.kv_attention(q, c, _dev(table), _dev(lengths), _dev(cu), new, most_kv, causal=True, return_lse=True)
    _check(h3, q, c, table, lengths, cu, out, lse, causal=True)


def test_segments_of_more_pages_than_a_part_holds(h3):
    """4 million keys of 8 heads in pages of 16: the table names each of 700 pages thousands of times, so that the
    definition is a softmax over 700 pages with their counts."""
    rng = np.random.default_rng(6)
    pages, page, heads, dim, L = 700, 16, 8, 128, 4_194_304 - 5
    c = _filled(h3, rng, np.arange(pages, dtype=np.int32)[None], [pages * page], pages, heads, page, dim)
    table = rng.integers(0, pages, (1, -(-L // page))).astype(np.int32)
    table[0, -1] = 3                                          # the page of the last, partly seen
    q = torch.randn(1, heads, dim, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    out, lse = _run(h3, q, c, table, [L], [0, 1], 1)
    counts = np.bincount(table[0, :-1], minlength=pages)[:, None].repeat(page, 1)
    counts[3, :L % page] += 1
    k, v = [O.cache_values(t.cpu().numpy(), s.cpu().numpy()) for t, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))]
    qv = q.double().cpu().numpy()[0]
    scale = dim ** -0.5
    for h in range(heads):
        kk, vv, n = k[:, h].reshape(-1, dim), v[:, h].reshape(-1, dim), counts.reshape(-1)
        s = kk @ qv[h] * scale
        w = np.exp(s - s.max())
        total = (w * n).sum()
        ref = (w * n) @ vv / total
        A, T = (w * n) @ np.abs(vv) / total, np.abs(w[:, None] * vv).max() / total
        e = 2.0 ** -17 * (scale * np.abs(kk * qv[h]).sum(1)).max()
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 4 * e) * A + L * 2.0 ** -22 * T
        assert (np.abs(out[0, h].double().cpu().numpy() - ref) <= tol).all()
        want = math.log(total) + s.max()
        assert abs(float(lse[0, h]) - want) <= e + 2.0 ** -20 * (1 + abs(want))
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("new", [1, 100])
def test_codes_past_32_bits(h3, new):
    """The same pages at the start of a small cache and at the end of one of 4.3 GB give the same bits."""
    rng = np.random.default_rng(5)
    L, page, heads, dim, many = 700, 128, 8, 128, 33_000
    table, pages = _tables(rng, [L], page)
    small = _filled(h3, rng, table, [L], pages, heads, page, dim)
    large = h3.KVCache.empty(many, page, heads, dim)
    for a, b in ((small.k_codes, large.k_codes), (small.v_codes, large.v_codes), (small.k_scale, large.k_scale),
                 (small.v_scale, large.v_scale)):
        b[many - pages:] = a
    assert large.k_codes.numel() > 2 ** 32
    q = torch.randn(new, heads, dim, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    want = _run(h3, q, small, table, [L], [0, new], new, causal=True)
    got = _run(h3, q, large, table + (many - pages), [L], [0, new], new, causal=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert h3.h3fp4_device_error() == 0
