"""Attention over the 8-bit paged cache against the 64-bit definition.

Bound per output, with A the softmax-weighted mean of |v|, P the largest
softmax_scale * sum |q k| and T the largest single |p v| / sum p of the row:
  2^-8 |out|           rounding to bf16 (half an ulp)
  2^-10 A              weights rounded to FP16 (2^-11), and their sum's and the product's FP32 roundings
  4 e A, e = 2^-17 P   scores: at most 128 FP32 additions (2^-24 each) on each of two exponents
  n 2^-22 T            weights below FP16's normal range: 2^-25 of the largest weight times 448 of its page's
                       scale, where T holds a code of at least 56
lse: e + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_cache import _dev, _patterns, _tables

pytestmark = pytest.mark.gpu


def _filled(h3, rng, table, lengths, pages, heads, page, dim, spread=2, stale_nan=True):
    """A cache whose used tokens are ordinary values and whose other bytes are leftovers, NaN codes among them."""
    c = h3.KVCache.empty(pages, page, heads, dim)
    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        x = O.e4m3_encode(rng.standard_normal(codes.shape) * 40)
        junk = np.full(codes.shape, 0x7F, dtype=np.uint8) if stale_nan else x
        used = np.zeros((pages, page), dtype=bool)
        for b, n in enumerate(lengths):
            pos = np.arange(n)
            used[table[b, pos // page], pos % page] = True
        codes.copy_(_dev(np.where(used[:, None, :, None], x, junk), torch.uint8))
        scale.copy_(torch.from_numpy(2.0 ** rng.integers(-6, -6 + spread, scale.shape)).float())
    return c


def _run(h3, q, c, table, lengths, cu, most, **kw):
    out, lse = h3.kv_attention(q, c, _dev(table), _dev(lengths), _dev(cu), most, max(list(lengths) + [0]), return_lse=True,
                               **kw)
    return out, lse


def _check(h3, q, c, table, lengths, cu, out, lse, scale=None, causal=False, window=0, rows=None):
    kv, vv = [O.cache_values(t.cpu().numpy(), s.cpu().numpy()) for t, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))]
    qv, got, gl = O.bf16_values(_patterns(q)), O.bf16_values(_patterns(out)), lse.cpu().numpy()
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for b in range(len(lengths)):
        L = int(lengths[b])
        k, v = O.gather(kv, table[b], L), O.gather(vv, table[b], L)
        n = int(cu[b + 1] - cu[b])
        ref, rl, A, P, T = O.attention(qv[cu[b]:cu[b + 1]], k, v, scale, causal, window)
        sel = np.arange(n) if rows is None else np.array([r for r in rows if r < n])
        g, gl_b = got[cu[b]:cu[b + 1]], gl[cu[b]:cu[b + 1]]
        e = 2.0 ** -17 * P
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 4 * e[..., None]) * A + L * 2.0 ** -22 * T[..., None] + 1e-38
        nan = np.isnan(ref)
        assert np.array_equal(np.isnan(g[sel]), nan[sel]), (b, int(np.isnan(g).sum()), int(nan.sum()))
        bad = ~(np.abs(g - ref) <= tol) & ~nan
        assert not bad[sel].any(), (b, int(bad[sel].sum()), float((np.abs(g - ref) / tol)[sel][~nan[sel]].max()))
        empty = rl == -np.inf
        assert np.array_equal(gl_b == -np.inf, empty)
        fine = ~empty & ~np.isnan(rl)
        assert (np.abs(gl_b[fine] - rl[fine]) <= e[fine] + 2.0 ** -20 * (1 + np.abs(rl[fine]))).all()
        assert np.isnan(gl_b[np.isnan(rl)]).all()
        assert (g[empty] == 0).all()


CASES = [   # (new, keys) of each sequence, heads, kv_heads, dim, page, causal, window
    ([(1, 1)], 1, 1, 128, 16, 1, 0),
    ([(1, 777)], 7, 7, 128, 16, 1, 0),
    ([(1, 16), (1, 17), (1, 15), (1, 300), (1, 0)], 8, 1, 64, 16, 1, 0),
    ([(1, 1000), (1, 33)], 16, 2, 128, 64, 0, 0),
    ([(1, 513)], 40, 8, 128, 128, 1, 100),
    ([(3, 200), (0, 50), (2, 2)], 6, 2, 128, 32, 1, 0),
    ([(5, 3), (4, 0), (1, 4)], 4, 4, 64, 16, 1, 0),          # more queries than keys: rows that see nothing
    ([(16, 129)], 5, 1, 64, 32, 1, 7),
    ([(20, 140), (33, 33)], 12, 3, 128, 64, 0, 0),
    ([(70, 70), (129, 400)], 4, 2, 128, 16, 1, 0),
    ([(257, 259)], 2, 2, 64, 128, 1, 50),
    ([(130, 513), (1, 90)], 3, 1, 128, 64, 0, 130),
    ([(300, 200)], 2, 1, 128, 64, 1, 0),
    ([(128, 128), (256, 384), (64, 1)], 2, 2, 128, 128, 0, 0),
    ([(200, 650)], 3, 3, 64, 16, 1, 1),                      # every query sees itself alone
]


@pytest.mark.parametrize("seqs,heads,kv_heads,dim,page,causal,window", CASES)
def test_against_64_bits(h3, seqs, heads, kv_heads, dim, page, causal, window):
    rng = np.random.default_rng(len(seqs) * 100 + heads)
    new, lengths = [a for a, _ in seqs], [b for _, b in seqs]
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, kv_heads, page, dim)
    cu = np.cumsum([0] + new)
    wide = torch.randn(cu[-1], heads + 2, dim, generator=torch.Generator().manual_seed(heads)).mul(2).bfloat16().cuda()
    q = wide[:, 1:1 + heads]
    out, lse = _run(h3, q, c, table, lengths, cu, max(new), causal=bool(causal), window=window)
    _check(h3, q, c, table, lengths, cu, out, lse, causal=bool(causal), window=window)
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("new,length", [(1, 20_011), (1, 4_099), (9, 3_000), (150, 5_003)])
def test_long_caches(h3, new, length):
    rng = np.random.default_rng(new)
    table, pages = _tables(rng, [length], 64)
    c = _filled(h3, rng, table, [length], pages, 2, 64, 128, spread=5)
    q = torch.randn(new, 4, 128, generator=torch.Generator().manual_seed(new)).mul(3).bfloat16().cuda()
    for causal in (False, True):
        out, lse = _run(h3, q, c, table, [length], [0, new], new, causal=causal)
        _check(h3, q, c, table, [length], [0, new], out, lse, causal=causal)


@pytest.mark.parametrize("new", [1, 150])
def test_query_sizes_and_scales(h3, new):
    """Rows of very large, very small and zero queries, a caller's softmax scale of either sign and zero, caches whose
    pages differ by 2^40 in scale, and scales that are no power of two."""
    rng = np.random.default_rng(3)
    L, page = 300, 32
    table, pages = _tables(rng, [L], page)
    q = torch.randn(new, 6, 128, generator=torch.Generator().manual_seed(5)).cuda()
    q *= torch.tensor([1.0, 1e4, 1e-20, 0.0, 3e-5, 100.0], device="cuda")[None, :, None]
    q[:, 5, 1:] *= 1e-6                                      # one channel far above the others
    q = q.bfloat16()
    for spread, factor, scale in ((2, 1.0, None), (40, 1e-6, None), (3, 1.7, -0.3), (3, 1.3, 0.0)):
        c = _filled(h3, rng, table, [L], pages, 2, page, 128, spread=spread)
        c.k_scale.mul_(min(1.0, factor))
        if factor > 1:
            c.v_scale.mul_(factor)
            c.k_scale.mul_(factor)
        kw = {} if scale is None else {"scale": scale}
        out, lse = _run(h3, q, c, table, [L], [0, new], new, **kw)
        _check(h3, q, c, table, [L], [0, new], out, lse, **kw)


@pytest.mark.parametrize("new,window", [(1, 0), (7, 0), (7, 9), (200, 0), (200, 60)])
def test_nan_reaches_only_those_that_see_it(h3, new, window):
    """NaN codes in keys and values of single tokens: rows that see the token get NaN (a key: everywhere, a value: in its
    channel), the others nothing, also where the token shares their tile."""
    rng = np.random.default_rng(4)
    L, page = 300, 16
    table, pages = _tables(rng, [L], page)
    c = _filled(h3, rng, table, [L], pages, 2, page, 128)
    for pos, head, kv, chan in ((L - 1, 0, 1, 5), (L - 3, 0, 1, 77), (L - 2, 1, 0, 9), (L - 100, 0, 1, 6), (100, 1, 1, 127)):
        codes = c.k_codes if kv == 0 else c.v_codes
        codes[int(table[0, pos // page]), head, pos % page, chan] = 0xFF if chan == 77 else 0x7F
    q = torch.randn(new, 4, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    out, lse = _run(h3, q, c, table, [L], [0, new], new, causal=True, window=window)
    _check(h3, q, c, table, [L], [0, new], out, lse, causal=True, window=window)


@pytest.mark.parametrize("new", [1, 140])
def test_nonfinite_queries_stay_in_their_row(h3, new):
    rng = np.random.default_rng(9)
    L, page = 90, 32
    table, pages = _tables(rng, [L], page)
    c = _filled(h3, rng, table, [L], pages, 2, page, 64)
    q = torch.randn(new, 4, 64, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    clean = _run(h3, q, c, table, [L], [0, new], new)[0]
    q[0, 1, 3], q[0, 2, 5] = float("nan"), float("inf")
    out = _run(h3, q, c, table, [L], [0, new], new)[0]
    assert out[0, 1].isnan().all() and out[0, 2].isnan().all()
    keep = torch.ones(new, 4, dtype=torch.bool)
    keep[0, 1] = keep[0, 2] = False
    assert torch.equal(out[keep.cuda()], clean[keep.cuda()])


@pytest.mark.parametrize("new", [1, 140])
def test_streams_outputs_and_repeats(h3, new):
    """Another stream, a strided output with canaries, no lse, and the same bits every time."""
    rng = np.random.default_rng(10)
    L, page = 2_000, 64
    table, pages = _tables(rng, [L, 40], page)
    c = _filled(h3, rng, table, [L, 40], pages, 2, page, 128)
    cu = [0, new, 2 * new]
    q = torch.randn(2 * new, 8, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    out, lse = _run(h3, q, c, table, [L, 40], cu, new, causal=True)
    args = q, c, _dev(table), _dev([L, 40]), _dev(cu), new, L
    wide = torch.full((2 * new, 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _, none = h3.kv_attention(*args, causal=True, out=wide[:, 1:9])
    s.synchronize()
    assert none is None and torch.equal(wide[:, 1:9], out)
    assert (wide[:, 0] == 7).all() and (wide[:, 9] == 7).all()
    for _ in range(3):
        assert torch.equal(h3.kv_attention(*args, causal=True)[0], out)


def test_captured_decoding_step_follows_lengths_on_the_device(h3):
    """A graph of write and attention replayed with other lengths and pages in the same buffers."""
    rng = np.random.default_rng(12)
    heads, dim, page, most = 4, 64, 16, 200
    table, pages = _tables(rng, [most, most], page)
    c = _filled(h3, rng, table, [most, most], pages, heads, page, dim)
    fresh = [t.clone() for t in (c.k_codes, c.k_scale, c.v_codes, c.v_scale)]
    tab, held, total, cu = _dev(table), _dev([30, 77]), _dev([31, 78]), _dev([0, 1, 2])
    x = torch.randn(2, 3 * heads, dim, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, k, v = x[:, :heads], x[:, heads:2 * heads], x[:, 2 * heads:]
    out = torch.empty(2, heads, dim, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(h3.h3fp4_kv_attention_workspace(2, heads, heads, dim, 2, 1, most) + 16, dtype=torch.uint8, device="cuda")

    def step():
        h3.kv_cache_write(c, k, v, tab, held, cu, 1)
        h3.kv_attention(q, c, tab, total, cu, 1, most, causal=True, out=out, workspace=ws)

    def reset():
        for t, u in zip((c.k_codes, c.k_scale, c.v_codes, c.v_scale), fresh):
            t.copy_(u)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for lens in ([30, 77], [0, 199], [150, 3]):
        held.copy_(_dev(lens))
        total.copy_(_dev([n + 1 for n in lens]))
        reset()
        step()
        want = out.clone()
        reset()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("new", [1, 140])
def test_out_of_range_entries_are_reported(h3, new):
    rng = np.random.default_rng(8)
    c = _filled(h3, rng, np.array([[0, 1]]), [32], 2, 2, 16, 64)
    q = torch.ones(new, 2, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(table=[[0, 2]]), dict(table=[[-7, 1]]), dict(len=[33]), dict(len=[-1]), dict(cu=[0, new + 1]),
               dict(cu=[1, 0]), dict(len=[2**31 - 1])):
        h3.kv_attention(q, c, _dev(kw.get("table", [[0, 1]])), _dev(np.array(kw.get("len", [32]), dtype=np.int64)),
                        _dev(kw.get("cu", [0, new])), new, 32)
        assert h3.h3fp4_device_error() == 512, kw
    h3.kv_attention(q, c, _dev([[0, 1]]), _dev([32]), _dev([0, new]), new, 32)
    assert h3.h3fp4_device_error() == 0
