"""Attention under a window whose first tokens stay visible, against the 64-bit
definition.  Bounds as for the attention without them."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_attention import _filled
from test_gpu_kv_cache import _dev, _patterns, _tables

pytestmark = pytest.mark.gpu


def check_rows(q, k, v, out, lse, scale, L, **seen):
    """One sequence's rows against the definition: the bounds of test_gpu_kv_attention."""
    ref, rl, A, P, T = O.attention(q, k, v, scale, **seen)
    e = 2.0 ** -17 * P
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 4 * e[..., None]) * A + L * 2.0 ** -22 * T[..., None] + 1e-38
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(out), nan), (int(np.isnan(out).sum()), int(nan.sum()))
    bad = ~(np.abs(out - ref) <= tol) & ~nan
    assert not bad.any(), (int(bad.sum()), float((np.abs(out - ref) / tol)[~nan].max()))
    empty, fine = rl == -np.inf, np.isfinite(rl)
    assert np.array_equal(lse == -np.inf, empty) and (out[empty] == 0).all()
    assert (np.abs(lse[fine] - rl[fine]) <= e[fine] + 2.0 ** -20 * (1 + np.abs(rl[fine]))).all()


def _check(c, q, table, lengths, cu, out, lse, **seen):
    kv, vv = [O.cache_values(t.cpu().numpy(), s.cpu().numpy()) for t, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))]
    qv, got, gl = O.bf16_values(_patterns(q)), O.bf16_values(_patterns(out)), lse.cpu().numpy()
    for b, L in enumerate(lengths):
        at = slice(int(cu[b]), int(cu[b + 1]))
        check_rows(qv[at], O.gather(kv, table[b], L), O.gather(vv, table[b], L), got[at], gl[at], q.shape[2] ** -0.5, L, **seen)


def _run(h3, q, c, table, lengths, cu, most, **kw):
    return h3.kv_attention(q, c, _dev(table), _dev(lengths), _dev(cu), most, max(list(lengths) + [0]), return_lse=True, **kw)


def _give_up(table, page, seqs, window, sinks):
    """Entries of pages of which no query sees anything, out of range."""
    t = table.copy()
    for b, (n, L) in enumerate(seqs):
        for p in range(-(-L // page)):
            if p * page >= sinks and (p + 1) * page <= max(0, L - n - window + 1):
                t[b, p] = 10 ** 6 if p % 2 else -5
    return t


CASES = [   # (new, keys) of each sequence, heads, kv_heads, dim, page, causal, window, sinks
    ([(1, 1)], 1, 1, 128, 16, 1, 5, 3),
    ([(1, 777)], 7, 7, 128, 16, 1, 100, 1),
    ([(1, 777)], 7, 7, 128, 128, 1, 1, 40),
    ([(1, 3000), (1, 40), (1, 900)], 16, 2, 128, 64, 1, 130, 70),
    ([(1, 300), (1, 16), (1, 0)], 8, 1, 64, 16, 1, 20, 4),
    ([(1, 300), (1, 16), (1, 33)], 8, 1, 64, 16, 0, 20, 24),
    ([(3, 500), (0, 50), (2, 2)], 6, 2, 128, 32, 1, 33, 17),
    ([(16, 1029)], 5, 1, 64, 32, 1, 7, 64),
    ([(20, 2140), (33, 33)], 12, 3, 128, 64, 0, 77, 129),
    ([(5, 3), (4, 0), (1, 4)], 4, 4, 64, 16, 1, 2, 1),       # more queries than keys
    ([(70, 70), (129, 1400)], 4, 2, 128, 16, 1, 60, 300),
    ([(257, 1259)], 2, 2, 64, 128, 1, 50, 5),
    ([(130, 1513), (1, 90)], 3, 1, 128, 64, 0, 130, 128),
    ([(300, 200)], 2, 1, 128, 64, 1, 9, 2),
    ([(200, 650)], 3, 3, 64, 16, 1, 1, 1),
    ([(200, 2650)], 3, 3, 128, 32, 1, 400, 900),             # sinks reach past several steps
    ([(140, 700)], 2, 2, 128, 64, 1, 100, 100_000),          # sinks past the end: the window hides nothing
    ([(9, 700)], 2, 2, 128, 64, 1, 100, 690),
]


@pytest.mark.parametrize("seqs,heads,kv_heads,dim,page,causal,window,sinks", CASES)
def test_against_64_bits(h3, seqs, heads, kv_heads, dim, page, causal, window, sinks):
    """Hidden tokens hold NaN, hidden pages are none."""
    rng = np.random.default_rng(len(seqs) * 100 + heads)
    new, lengths = [a for a, _ in seqs], [b for _, b in seqs]
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, kv_heads, page, dim)
    for b, (n, L) in enumerate(seqs):
        for pos in range(min(sinks, L), max(0, L - n - window + 1)):
            for codes in (c.k_codes, c.v_codes):
                codes[int(table[b, pos // page]), :, pos % page] = 0x7F
    cu = np.cumsum([0] + new)
    wide = torch.randn(cu[-1], heads + 2, dim, generator=torch.Generator().manual_seed(heads)).mul(2).bfloat16().cuda()
    q = wide[:, 1:1 + heads]
    out, lse = _run(h3, q, c, _give_up(table, page, seqs, window, sinks), lengths, cu, max(new), causal=bool(causal), window=window,
                    sinks=sinks)
    assert h3.h3fp4_device_error() == 0
    _check(c, q, table, lengths, cu, out, lse, causal=bool(causal), window=window, sinks=sinks)


@pytest.mark.parametrize("new,length,window,sinks", [(1, 40_011, 9_000, 100), (1, 20_000, 50, 8_000), (9, 9_000, 3_000, 5),
                                                     (150, 9_003, 2_000, 700), (700, 5_000, 100, 1_000)])
def test_long_caches(h3, new, length, window, sinks):
    rng = np.random.default_rng(new)
    table, pages = _tables(rng, [length], 64)
    c = _filled(h3, rng, table, [length], pages, 2, 64, 128, spread=5)
    q = torch.randn(new, 4, 128, generator=torch.Generator().manual_seed(new)).mul(3).bfloat16().cuda()
    for causal in (False, True):
        out, lse = _run(h3, q, c, table, [length], [0, new], new, causal=causal, window=window, sinks=sinks)
        _check(c, q, table, [length], [0, new], out, lse, causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("new", [1, 7, 200])
def test_nan_reaches_only_those_that_see_it(h3, new):
    rng = np.random.default_rng(4)
    L, page, window, sinks = 700, 16, 150, 40
    table, pages = _tables(rng, [L], page)
    c = _filled(h3, rng, table, [L], pages, 2, page, 128)
    for pos, head, kv, chan in ((L - 1, 0, 1, 5), (3, 0, 1, 77), (39, 1, 1, 9), (40, 1, 1, 10), (L - 160, 0, 1, 6), (L - 200, 0, 0, 127)):
        codes = c.k_codes if kv == 0 else c.v_codes
        codes[int(table[0, pos // page]), head, pos % page, chan] = 0x7F
    q = torch.randn(new, 4, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    out, lse = _run(h3, q, c, table, [L], [0, new], new, causal=True, window=window, sinks=sinks)
    _check(c, q, table, [L], [0, new], out, lse, causal=True, window=window, sinks=sinks)


@pytest.mark.parametrize("new", [1, 5, 140])
def test_values_scales_far_apart(h3, new):
    """Sinks whose values' scale is 2^100 times the window's, and the other way round."""
    rng = np.random.default_rng(6)
    L, page = 900, 32
    table, pages = _tables(rng, [L], page)
    q = torch.randn(new, 2, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    for first, rest in ((60, -40), (-40, 60)):
        c = _filled(h3, rng, table, [L], pages, 1, page, 128)
        c.v_scale.fill_(2.0 ** rest)
        c.v_scale[int(table[0, 0])] = 2.0 ** first
        kw = dict(causal=True, window=200, sinks=20)
        out, lse = _run(h3, q, c, table, [L], [0, new], new, **kw)
        _check(c, q, table, [L], [0, new], out, lse, **kw)


@pytest.mark.parametrize("new", [1, 6, 140])
def test_without_a_window_or_sinks_it_is_the_attention_without(h3, new):
    rng = np.random.default_rng(9)
    L, page = 1_000, 64
    table, pages = _tables(rng, [L], page)
    c = _filled(h3, rng, table, [L], pages, 2, page, 128)
    q = torch.randn(new, 8, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    plain = _run(h3, q, c, table, [L], [0, new], new, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, _run(h3, q, c, table, [L], [0, new], new, causal=True, sinks=9)))
    under = _run(h3, q, c, table, [L], [0, new], new, causal=True, window=77)
    wide = torch.full((new, 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    need = h3.h3fp4_kv_attention_workspace(new, 8, 2, 128, 1, new, L)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    lse = torch.empty(new, 8, device="cuda")
    h3.h3fp4_kv_attention_sinks(q.data_ptr(), 1024, 128, wide[:, 1:].data_ptr(), 1280, 128, lse.data_ptr(), new, 8, c.struct(),
                                h3._kv_batch(t := _dev(table), n := _dev([L]), cu := _dev([0, new]), new, 0), L, 128 ** -0.5, 1, 77, 0,
                                ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(wide[:, 1:9], under[0]) and torch.equal(lse, under[1])
    assert (wide[:, 0] == 7).all() and (wide[:, 9] == 7).all()


@pytest.mark.parametrize("new", [1, 140])
@pytest.mark.parametrize("pages", [0, 3])
def test_sequences_without_keys(h3, new, pages):
    """No keys, of a cache with and without pages: zeros and minus infinity, nothing reported."""
    c = h3.KVCache.empty(pages, 32, 2, 128)
    q = torch.ones(new, 4, 128, dtype=torch.bfloat16, device="cuda")
    for most in (0, 90):
        out, lse = h3.kv_attention(q, c, torch.empty(1, 0, dtype=torch.int32, device="cuda"), _dev([0]), _dev([0, new]), new, most,
                                   causal=True, window=4, sinks=2, return_lse=True)
        assert (out == 0).all() and (lse == -np.inf).all()
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("new", [1, 7, 140])
def test_what_stands_in_for_hidden_pages_has_no_effect(h3, new):
    """Page 0, and everything past the end, holds NaN: a sequence that does not use it, with a gap of whole pages, pages that
    end inside a step, and a last step that is not full."""
    rng = np.random.default_rng(11)
    L, page = 1_111, 16
    table, pages = _tables(rng, [L], page)
    table = np.where(table == 0, pages, table)                      # page 0 goes unused
    c = _filled(h3, rng, table, [L], pages + 1, 2, page, 128)
    for codes in (c.k_codes, c.v_codes):
        codes[0] = 0x7F
    q = torch.randn(new, 4, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    for window, sinks in ((100, 10), (3, 200), (500, 129)):
        given = _give_up(table, page, [(new, L)], window, sinks)
        out, lse = _run(h3, q, c, given, [L], [0, new], new, causal=True, window=window, sinks=sinks)
        assert h3.h3fp4_device_error() == 0
        _check(c, q, table, [L], [0, new], out, lse, causal=True, window=window, sinks=sinks)


@pytest.mark.parametrize("new", [1, 140])
def test_codes_past_32_bits(h3, new):
    """The last pages of a cache of 5.2 GB of keys against the same pages in a small one, with sinks and behind a prefix."""
    rng = np.random.default_rng(12)
    L, page, heads = 700, 128, 8
    small = h3.KVCache.empty(6, page, heads, 128)
    for t in (small.k_codes, small.v_codes):
        t.copy_(_dev(O.e4m3_encode(rng.standard_normal(t.shape) * 40), torch.uint8))
    many = 40_000
    big = h3.KVCache.empty(many, page, heads, 128)
    for a, b in ((big.k_codes, small.k_codes), (big.v_codes, small.v_codes)):
        a[-6:].copy_(b)
    table = np.arange(6)[None]
    q = torch.randn(new, heads, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    got = []
    for c, first in ((small, 0), (big, many - 6)):
        t = _dev(table + first)
        got.append(h3.kv_attention(q, c, t, _dev([L]), _dev([0, new]), new, L, causal=True, window=100, sinks=200, return_lse=True))
        prefix = h3.SharedPrefix(t[:, :2].contiguous(), _dev([200]), _dev([0, new]), new, 200)
        got.append(h3.kv_attention_shared(q, c, prefix, t[:, 2:].contiguous(), _dev([300]), _dev([0, new]), new, 300, return_lse=True))
    for a, b in zip(got[:2], got[2:]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("batch,kv_heads,dim,window,sinks", [(36, 8, 128, 900, 70), (29, 8, 64, 700, 33), (300, 1, 128, 40, 4_000), (150, 1, 128, 600, 9),
                                                             (700, 1, 64, 300, 5), (12, 20, 128, 1_500, 1)])
def test_batches_whose_rows_have_ctas_to_themselves(h3, batch, kv_heads, dim, window, sinks):
    """Ragged batches of every size about the number of SMs, whose rows go to one CTA each (of four or six warps) or a few:
    sampled sequences against the definition, all against calls of few sequences."""
    rng = np.random.default_rng(batch)
    lengths = [int(n) for n in rng.integers(1, 2_600, batch)]
    lengths[0], lengths[1] = 2_600, 1
    page, heads = 32, 2 * kv_heads
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, kv_heads, page, dim)
    q = torch.randn(batch, heads, dim, generator=torch.Generator().manual_seed(batch)).mul(2).bfloat16().cuda()
    given = _give_up(table, page, [(1, L) for L in lengths], window, sinks)
    kw = dict(causal=True, window=window, sinks=sinks)
    out, lse = _run(h3, q, c, given, lengths, np.arange(batch + 1), 1, **kw)
    assert h3.h3fp4_device_error() == 0
    for b in (0, 1, 2, batch // 2, batch - 1):
        one = _run(h3, q[b:b + 1], c, given[b:b + 1], lengths[b:b + 1], [0, 1], 1, **kw)
        _check(c, q[b:b + 1], table[b:b + 1], lengths[b:b + 1], [0, 1], out[b:b + 1], lse[b:b + 1], **kw)
        _check(c, q[b:b + 1], table[b:b + 1], lengths[b:b + 1], [0, 1], *one, **kw)
    for b in range(0, batch, 5):                       # the rest: two spreads of the same sums, each rounded to bf16 (2^-8)
        n = min(5, batch - b)
        few, few_lse = _run(h3, q[b:b + n], c, given[b:b + n], lengths[b:b + n], np.arange(n + 1), 1, **kw)
        scale = out[b:b + n].float().abs().amax(-1, keepdim=True)
        assert ((few.float() - out[b:b + n].float()).abs() <= 2.0 ** -7 * scale).all()
        assert torch.allclose(few_lse, lse[b:b + n], rtol=0, atol=1e-3)


@pytest.mark.parametrize("batch,heads,kv_heads,dim,n", [(1, 4, 1, 128, 1), (2, 8, 4, 128, 2), (1, 16, 2, 64, 1), (1, 96, 6, 128, 1), (1, 6, 2, 64, 4),
                                                        (3, 40, 8, 128, 2)])
def test_few_rows_over_many_keys_are_joined_from_many_parts(h3, batch, heads, kv_heads, dim, n):
    """Rows whose parts lie with hundreds of CTAs, joined a row, two rows or a whole tile at a time."""
    rng = np.random.default_rng(heads)
    lengths = [int(x) for x in rng.integers(14_000, 17_000, batch)]
    page = 64
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, kv_heads, page, dim)
    q = torch.randn(batch * n, heads, dim, generator=torch.Generator().manual_seed(heads)).mul(2).bfloat16().cuda()
    window, sinks = 9_000, 130
    given = _give_up(table, page, [(n, L) for L in lengths], window, sinks)
    kw = dict(causal=True, window=window, sinks=sinks)
    cu = np.arange(batch + 1) * n
    out, lse = _run(h3, q, c, given, lengths, cu, n, **kw)
    assert h3.h3fp4_device_error() == 0
    _check(c, q, table, lengths, cu, out, lse, **kw)


@pytest.mark.parametrize("new,heads", [(1, 4), (1, 32), (20, 4), (140, 4)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2_000, 0), (1_500, 70)])
def test_rows_of_a_refused_sequence_stay_as_they_were(h3, new, heads, window, sinks):
    """The middle one of three, whose pages or keys are past what was said, also where the parts of its keys would be joined."""
    rng = np.random.default_rng(new)
    page, lengths = 32, [2_900, 2_800, 2_700]
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, 2, page, 128)
    q = torch.randn(3 * new, heads, 128, generator=torch.Generator().manual_seed(new)).mul(2).bfloat16().cuda()
    cu, kw = np.arange(4) * new, dict(causal=True, window=window, sinks=sinks)
    for keys, most in ((page * table.shape[1] + 1, 20_000), (20_001, 20_000), (-1, 20_000)):
        out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], 5.0, device="cuda")
        need = h3.h3fp4_kv_attention_workspace(3 * new, heads, 2, 128, 3, new, most)
        ws = torch.full((max(16, need),), 0x40, dtype=torch.uint8, device="cuda")
        given = [lengths[0], keys, lengths[2]]
        h3.kv_attention(q, c, _dev(table), _dev(given), _dev(cu), new, most, out=out, lse=lse, workspace=ws, **kw)
        assert h3.h3fp4_device_error() == 512
        assert (out[new:2 * new] == 7).all() and (lse[new:2 * new] == 5).all()
        for b in (0, 2) if keys < 0 else ():
            at = slice(b * new, b * new + new)
            _check(c, q[at], table[b:b + 1], lengths[b:b + 1], [0, new], out[at], lse[at], **kw)


def _filled_on_gpu(h3, table, lengths, pages, heads, page, dim, seed):
    """As _filled: NaN wherever no sequence has a token."""
    c, gen = h3.KVCache.empty(pages, page, heads, dim), torch.Generator(device="cuda").manual_seed(seed)
    used = np.zeros((pages, page), dtype=bool)
    for b, n in enumerate(lengths):
        used[table[b, np.arange(n) // page], np.arange(n) % page] = True
    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        x = torch.randn(codes.shape, generator=gen, device="cuda").mul(40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.copy_(torch.where(torch.from_numpy(used).cuda()[:, None, :, None], x, torch.full_like(x, 0x7F)))
        scale.copy_(torch.exp2(torch.randint(-6, -4, scale.shape, generator=gen, device="cuda").float()))
    return c


def _all_within_bounds(c, q, table, lengths, out, lse, window, sinks):
    """check_rows' bounds for every sequence of one token each, the definition evaluated on the GPU in 64 bits."""
    heads, dim = q.shape[1:]
    group, page = heads // c.heads, c.page_size
    for b, L in enumerate(lengths):
        pos = torch.arange(L, device="cuda")
        pos = pos[(pos > L - 1 - window) | (pos < sinks)]
        ids = _dev(table[b], torch.int64)[pos // page]
        k, v = [(x[ids, :, pos % page].view(torch.float8_e4m3fn).double() * s[ids][..., None].double()).repeat_interleave(group, 1)
                for x, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))]
        mine = q[b].double()
        score = (mine * k).sum(2) * dim ** -0.5
        size = (mine * k).abs().sum(2).amax(0) * dim ** -0.5
        log, p = torch.logsumexp(score, 0), torch.softmax(score, 0)
        e = 2.0 ** -17 * size
        assert ((lse[b].double() - log).abs() <= e + 2.0 ** -20 * (1 + log.abs())).all(), b
        part = p[:, :, None] * v
        ref, near, top = part.sum(0), part.abs().sum(0), part.abs().amax(0)
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 4 * e[:, None]) * near + L * 2.0 ** -22 * top + 1e-38
        assert ((out[b].double() - ref).abs() <= tol).all(), b


@pytest.mark.parametrize("batch,kv_heads,dim,window,sinks", [(36, 8, 128, 900, 70), (29, 8, 64, 700, 33), (300, 1, 128, 40, 4_000), (150, 1, 128, 600, 9),
                                                             (700, 1, 64, 300, 5), (12, 20, 128, 1_500, 1)])
def test_every_sequence_of_batches_whose_rows_have_ctas_to_themselves(h3, batch, kv_heads, dim, window, sinks):
    rng = np.random.default_rng(batch + 1)
    lengths = [int(n) for n in rng.integers(1, 2_600, batch)]
    lengths[0], lengths[-1] = 2_600, 1
    table, pages = _tables(rng, lengths, 32)
    c = _filled_on_gpu(h3, table, lengths, pages, kv_heads, 32, dim, batch)
    q = torch.randn(batch, 2 * kv_heads, dim, generator=torch.Generator().manual_seed(batch)).mul(2).bfloat16().cuda()
    given = _give_up(table, 32, [(1, L) for L in lengths], window, sinks)
    out, lse = _run(h3, q, c, given, lengths, np.arange(batch + 1), 1, causal=True, window=window, sinks=sinks)
    assert h3.h3fp4_device_error() == 0
    _all_within_bounds(c, q, table, lengths, out, lse, window, sinks)
