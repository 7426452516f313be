"""The 8-bit paged cache: codes and scales bit for bit against the 64-bit
oracle (the definition rounds once, to E4M3), read-back exact, appends over
half-filled pages, non-finite values, range reports."""
import numpy as np
import pytest
import torch

from oracle import attention as O

pytestmark = pytest.mark.gpu


def _patterns(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _tables(rng, lengths, page, spare=2):
    counts = [-(-n // page) for n in lengths]
    ids = rng.permutation(sum(counts) + spare).astype(np.int32)
    table = np.full((len(lengths), max(1, max(counts))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(counts) + spare


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _cache(h3, rng, pages, heads, page, dim):
    """A cache full of leftovers, NaN codes and odd scales among them."""
    c = h3.KVCache.empty(pages, page, heads, dim)
    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        codes.copy_(_dev(rng.integers(0, 256, codes.shape), torch.uint8))
        scale.copy_(torch.from_numpy(2.0 ** rng.integers(-30, 30, scale.shape)).float())
    return c


CASES = [   # held and new tokens of each sequence, heads, dim, page
    ([0], [1], 1, 128, 16),
    ([0, 3, 15, 16], [1, 1, 1, 1], 8, 128, 16),
    ([5, 0, 64, 63], [100, 0, 1, 2], 3, 64, 64),
    ([0, 130], [257, 40], 2, 128, 128),
    ([31], [300], 5, 64, 32),
    ([7, 8, 9], [9, 8, 7], 56, 64, 16),
]


@pytest.mark.parametrize("held,new,heads,dim,page", CASES)
def test_write_bits_and_read_back(h3, held, new, heads, dim, page):
    rng = np.random.default_rng(page + heads)
    table, pages = _tables(rng, [a + b for a, b in zip(held, new)], page)
    c = _cache(h3, rng, pages, heads, page, dim)
    # earlier tokens are written first, so that half-filled pages hold real values of another size
    cu0, cu = np.cumsum([0] + held), np.cumsum([0] + new)
    tab = _dev(table)
    first = torch.randn(max(1, cu0[-1]), heads, dim, generator=torch.Generator().manual_seed(1)).mul(0.01).bfloat16().cuda()
    wide = torch.randn(max(1, cu[-1]), 3 * heads, dim, generator=torch.Generator().manual_seed(2))
    wide *= torch.exp2(torch.randint(-8, 8, (max(1, cu[-1]), 1, 1), generator=torch.Generator().manual_seed(3)).float())
    wide = wide.bfloat16().cuda()
    k, v = wide[:cu[-1], heads:2 * heads], wide[:cu[-1], 2 * heads:]
    want = [[t.cpu().numpy().copy() for t in (c.k_codes, c.k_scale)], [t.cpu().numpy().copy() for t in (c.v_codes, c.v_scale)]]
    zeros = np.zeros(len(held), dtype=np.int64)
    if cu0[-1]:
        h3.kv_cache_write(c, first, first, tab, _dev(zeros), _dev(cu0), max(held))
        for codes, scale in want:
            O.cache_write(codes, scale, O.bf16_values(_patterns(first)), table, zeros, cu0)
    h3.kv_cache_write(c, k, v, tab, _dev(held), _dev(cu), max(new))
    for (codes, scale), x in zip(want, (k, v)):
        O.cache_write(codes, scale, O.bf16_values(_patterns(x)), table, np.array(held), cu)
    for (codes, scale), (gc, gs) in zip(want, ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))):
        assert np.array_equal(gs.cpu().numpy(), scale)
        assert np.array_equal(gc.cpu().numpy(), codes)

    lengths = np.array(held) + np.array(new)
    back = np.cumsum([0] + list(lengths))
    ko, vo = h3.kv_cache_read(c, tab, None, _dev(back), int(back[-1]), int(max(lengths)))
    for (codes, scale), got in zip(want, (ko, vo)):
        val = O.cache_values(codes, scale)
        ref = np.concatenate([O.gather(val, table[b], int(lengths[b])) for b in range(len(held))])
        assert np.array_equal(O.bf16_values(_patterns(got)), ref)
    # a part, from a position inside a page, into a strided output
    start = np.array([min(3, max(0, n - 1)) for n in lengths])
    cu2 = np.cumsum([0] + list(lengths - start))
    out = torch.zeros(int(cu2[-1]), 2 * heads, dim, dtype=torch.bfloat16, device="cuda")
    h3.kv_cache_read(c, tab, _dev(start), _dev(cu2), int(cu2[-1]), int(max(lengths)), k=out[:, :heads], v=out[:, heads:])
    keep = np.concatenate([np.arange(back[b] + start[b], back[b + 1]) for b in range(len(held))])
    assert torch.equal(out[:, :heads], ko[_dev(keep, torch.int64)]) and torch.equal(out[:, heads:], vo[_dev(keep, torch.int64)])
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("layout,dims", [("interleaved", (32, 48, 48)), ("halves", (44, 42, 42)), ("halves", (20, 22))])
@pytest.mark.parametrize("page,held,new", [(64, 70, 200), (16, 3, 1), (128, 0, 129), (32, 31, 40)])
def test_rotated_write_equals_rotation_then_write(h3, layout, dims, page, held, new):
    heads, dim = 9, 128
    rng = np.random.default_rng(7)
    table, pages = _tables(rng, [held + new], page)
    a, b = _cache(h3, rng, pages, heads, page, dim), None
    b = h3.KVCache(*[t.clone() for t in (a.k_codes, a.k_scale, a.v_codes, a.v_scale)])
    g = torch.Generator().manual_seed(11)
    x = torch.randn(new, 2 * heads, dim, generator=g).bfloat16().cuda()
    pos = torch.rand(new, len(dims), generator=g).mul(500).floor().cuda()
    r = h3.Rope(pos, h3.rope_frequencies(dims), dims, layout=layout)
    tab, at, cu = _dev(table), _dev([held]), _dev([0, new])
    h3.kv_cache_write(a, x[:, :heads], x[:, heads:], tab, at, cu, new, rope=r)
    h3.kv_cache_write(b, h3.rope_axes(x[:, :heads], r), x[:, heads:], tab, at, cu, new)
    for s, t in ((a.k_codes, b.k_codes), (a.v_codes, b.v_codes), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert torch.equal(s, t)


def test_every_bf16_value_and_extreme_scales(h3):
    """Every bf16 pattern once, 2,048 of nearly one exponent a page and head, so that all scales occur."""
    dim, page, heads = 128, 16, 1
    bits = np.arange(65536, dtype=np.uint16)
    order = np.argsort((bits & 0x7FFF).astype(np.int32), kind="stable")
    bits = bits[order].reshape(-1, heads, dim)
    n = bits.shape[0]
    x = torch.from_numpy(bits.view(np.int16)).cuda()
    rng = np.random.default_rng(1)
    table, pages = _tables(rng, [n], page, spare=0)
    c = _cache(h3, rng, pages, heads, page, dim)
    codes, scale = c.k_codes.cpu().numpy().copy(), c.k_scale.cpu().numpy().copy()
    h3.kv_cache_write(c, x, x, _dev(table), _dev([0]), _dev([0, n]), n)
    O.cache_write(codes, scale, O.bf16_values(bits), table, np.array([0]), np.array([0, n]))
    assert np.array_equal(c.k_scale.cpu().numpy(), scale) and np.array_equal(c.v_scale.cpu().numpy(), scale)
    assert np.array_equal(c.k_codes.cpu().numpy(), codes) and np.array_equal(c.v_codes.cpu().numpy(), codes)
    k, _ = h3.kv_cache_read(c, _dev(table), None, _dev([0, n]), n, n)
    ref = O.gather(O.cache_values(codes, scale), table[0], n)
    got = O.bf16_values(_patterns(k))
    assert np.array_equal(got, ref, equal_nan=True)


def test_token_by_token_keeps_scales_and_repeats(h3):
    """33 single-token appends of growing and shrinking tokens, against the oracle; the last repeated changes nothing."""
    rng = np.random.default_rng(5)
    heads, dim, page, n = 2, 64, 32, 33
    table, pages = _tables(rng, [n], page)
    c = _cache(h3, rng, pages, heads, page, dim)
    codes, scale = c.v_codes.cpu().numpy().copy(), c.v_scale.cpu().numpy().copy()
    size = 2.0 ** rng.integers(-12, 12, n)
    size[0] = 0.0                                          # an all-zero token first: the smallest scale
    x = (rng.standard_normal((n, heads, dim)) * size[:, None, None]).astype(np.float32)
    xt = torch.from_numpy(x).bfloat16().cuda()
    for i in range(n):
        h3.kv_cache_write(c, xt[i:i + 1], xt[i:i + 1], _dev(table), _dev([i]), _dev([0, 1]), 1)
        O.cache_write(codes, scale, O.bf16_values(_patterns(xt[i:i + 1])), table, np.array([i]), np.array([0, 1]))
    assert np.array_equal(c.v_scale.cpu().numpy(), scale) and np.array_equal(c.v_codes.cpu().numpy(), codes)
    h3.kv_cache_write(c, xt[n - 1:], xt[n - 1:], _dev(table), _dev([n - 1]), _dev([0, 1]), 1)
    assert np.array_equal(c.v_scale.cpu().numpy(), scale) and np.array_equal(c.v_codes.cpu().numpy(), codes)


def test_a_callers_own_scale(h3):
    """A half-filled page whose scale is no power of two: kept where it suffices, else replaced, both rounded once."""
    rng = np.random.default_rng(6)
    heads, dim, page = 2, 64, 16
    for own in (0.3, 1e-3):
        c = _cache(h3, rng, 1, heads, page, dim)
        c.k_codes.copy_(_dev(rng.integers(0, 0x7F, c.k_codes.shape), torch.uint8))
        c.k_scale.fill_(own)
        codes, scale = c.k_codes.cpu().numpy().copy(), c.k_scale.cpu().numpy().copy()
        x = torch.randn(5, heads, dim, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
        h3.kv_cache_write(c, x, x, _dev([[0]]), _dev([4]), _dev([0, 5]), 5)
        O.cache_write(codes, scale, O.bf16_values(_patterns(x)), np.array([[0]]), np.array([4]), np.array([0, 5]))
        assert np.array_equal(c.k_scale.cpu().numpy(), scale)
        # a quotient by such a scale is rounded to FP32 before E4M3: codes may differ where that meets a midpoint
        assert (c.k_codes.cpu().numpy() != codes).mean() < 1e-3


def test_out_of_range_entries_are_reported_and_not_followed(h3):
    rng = np.random.default_rng(8)
    heads, dim, page = 2, 64, 16
    c = _cache(h3, rng, 4, heads, page, dim)
    before = [t.clone() for t in (c.k_codes, c.k_scale, c.v_codes, c.v_scale)]
    x = torch.ones(8, heads, dim, dtype=torch.bfloat16, device="cuda")
    bad = [dict(table=[[4]]), dict(table=[[-1]]), dict(held=[16]), dict(held=[-1]), dict(cu=[0, 9]), dict(cu=[4, 2]),
           dict(most=3), dict(held=[2**31 - 1]), dict(cu=[-2, 4])]
    for kw in bad:
        t, held = _dev(kw.get("table", [[1]])), _dev(np.array(kw.get("held", [0]), dtype=np.int64))
        cu, most = _dev(kw.get("cu", [0, 8])), kw.get("most", 8)
        h3.kv_cache_write(c, x, x, t, held, cu, most)
        assert h3.h3fp4_device_error() == 512, kw
        out = torch.zeros(8, heads, dim, dtype=torch.bfloat16, device="cuda")
        h3.kv_cache_read(c, t, held, cu, 8, most, k=out, v=out.clone())
        assert h3.h3fp4_device_error() == 512, kw
        assert not out.any()
    for t, u in zip((c.k_codes, c.k_scale, c.v_codes, c.v_scale), before):
        assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))
    assert h3.h3fp4_device_error() == 0


def test_cache_offsets_past_32_bits(h3):
    """A page whose codes start past 2^32 bytes."""
    heads, dim, page = 8, 128, 128
    pages = 2**32 // (heads * dim * page) + 3
    c = h3.KVCache.empty(pages, page, heads, dim)
    x = torch.randn(200, heads, dim, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    small = h3.KVCache.empty(2, page, heads, dim)
    args = _dev([0]), _dev([0, 200]), 200
    h3.kv_cache_write(c, x, x, _dev([[pages - 1, pages - 3]]), *args)
    h3.kv_cache_write(small, x, x, _dev([[0, 1]]), *args)
    a = h3.kv_cache_read(c, _dev([[pages - 1, pages - 3]]), None, _dev([0, 200]), 200, 200)
    b = h3.kv_cache_read(small, _dev([[0, 1]]), None, _dev([0, 200]), 200, 200)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
