"""The 8-bit paged cache and its attention at the edges of what their arguments
may hold.  Bounds as in test_gpu_kv_attention where a test gives none of its own."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_attention import _check, _filled, _run
from test_gpu_kv_cache import _dev, _tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 16, 140])
def test_a_cache_without_pages(h3, new):
    """No page exists: a length above zero is out of range and nothing is read, a length of zero sees nothing."""
    c = h3.KVCache.empty(0, 16, 2, 64)
    q = torch.ones(new, 4, 64, dtype=torch.bfloat16, device="cuda")
    for table, length, max_kv in (([[0, 0]], 32, 32), ([[0] * 64], 1_024, 1_024), ([[0] * 64], 1_000, 1 << 20)):
        h3.kv_attention(q, c, _dev(table), _dev([length]), _dev([0, new]), new, max_kv)
        assert h3.h3fp4_device_error() == 512, (length, max_kv)
    for table in ([[0, 0]], [[-1]]):
        out, lse = h3.kv_attention(q, c, _dev(table), _dev([0]), _dev([0, new]), new, 32, return_lse=True)
        assert not out.any() and (lse == -float("inf")).all()
        assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("new", [1, 140])
@pytest.mark.parametrize("size,scale,log_k_scale", [
    (1.0, 0.0, -58), (1.0, 0.0, 100),          # a scale of zero: the mean of what is seen, whatever the keys hold
    (1e-25, None, -58),                        # every score nearly zero
    (1e-30, None, 91), (1e-30, None, 96),      # very small queries against very large keys: scores of ordinary size
    (1.0, 1e-30, 95),
    (1e20, None, -58),                         # and the other way round
])
def test_factors_far_from_one(h3, new, size, scale, log_k_scale):
    """Causal, with a ragged tail, so that hidden keys share steps with visible ones."""
    rng = np.random.default_rng(21)
    lengths, page = [300, 181], 32
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, 2, page, 128)
    c.k_scale.fill_(2.0 ** log_k_scale)
    cu = [0, new, 2 * new]
    q = torch.randn(2 * new, 4, 128, generator=torch.Generator().manual_seed(8)).mul(size).bfloat16().cuda()
    kw = {} if scale is None else {"scale": scale}
    out, lse = _run(h3, q, c, table, lengths, cu, new, causal=True, **kw)
    _check(h3, q, c, table, lengths, cu, out, lse, causal=True, **kw)
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("most", [1, 16, 140])
def test_a_sequence_without_queries_is_not_looked_at(h3, most):
    """An idle slot of a batch, whatever its length and its row of the table hold, is no error in either kernel."""
    rng = np.random.default_rng(22)
    lengths, page = [64, 64, 50], 16
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, 2, page, 64)
    cu = [0, most, most, most + 1]
    q = torch.randn(most + 1, 4, 64, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    want = h3.kv_attention(q, c, _dev(table), _dev(lengths), _dev(cu), most, 64, causal=True)[0]
    for idle in (0, 65, 10_000, 2**31 - 1, -3):
        table[1] = -1
        got = h3.kv_attention(q, c, _dev(table), _dev(np.array([64, idle, 50])), _dev(cu), most, 64, causal=True)[0]
        assert torch.equal(got, want)
        assert h3.h3fp4_device_error() == 0, idle


def test_a_sequence_without_tokens_is_not_looked_at_by_the_cache(h3):
    rng = np.random.default_rng(23)
    table, pages = _tables(rng, [20, 20, 20], 16)
    x = torch.randn(9, 2, 64, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    cu = _dev([0, 5, 5, 9])
    caches = [h3.KVCache.empty(pages, 16, 2, 64) for _ in range(2)]
    table[1] = -1
    for idle, c in ((0, caches[0]), (10_000, caches[1]), (2**31 - 1, caches[1]), (-3, caches[1])):
        held = _dev(np.array([0, idle, 0]))
        h3.kv_cache_write(c, x, x, _dev(table), held, cu, 5)
        got = h3.kv_cache_read(c, _dev(table), held, cu, 9, 5)
        want = h3.kv_cache_read(caches[0], _dev(table), _dev([0, 0, 0]), cu, 9, 5)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert h3.h3fp4_device_error() == 0, idle


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("new,heads", [(1, 2), (3, 8), (9, 4), (140, 2)])
def test_pages_before_a_window_may_be_given_up(h3, new, heads, page):
    """Table entries before all that the queries see hold anything: the same bits and no report."""
    rng = np.random.default_rng(24)
    lengths = [1_200, 777]
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, 2, page, 64)
    cu = [0, new, 2 * new]
    q = torch.randn(2 * new, heads, 64, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    for window in (1, 5, 17, 33, 40, 100, 129, 500):
        for causal in (True, False):
            want, lse = _run(h3, q, c, table, lengths, cu, new, causal=causal, window=window)
            _check(h3, q, c, table, lengths, cu, want, lse, causal=causal, window=window)
            freed = table.copy()
            for b, n in enumerate(lengths):
                gone = max(0, n - new - window + 1) // page      # whole pages before the first query's window
                freed[b, :gone] = rng.choice([-1, pages, 2**31 - 1], gone)
            got = h3.kv_attention(q, c, _dev(freed), _dev(lengths), _dev(cu), new, max(lengths), causal=causal, window=window)[0]
            assert torch.equal(got, want)
            assert h3.h3fp4_device_error() == 0, (window, causal)


@pytest.mark.parametrize("gap", [0, 40])
@pytest.mark.parametrize("order", ["turn by turn", "small ones first", "large ones first"])
@pytest.mark.parametrize("new,length", [(1, 90), (1, 300), (9, 300), (140, 300), (1, 9_000), (20, 4_000), (140, 2_500)])
def test_value_scales_far_apart(h3, new, length, order, gap):
    """Pages whose values' scales are those of an all-zero page (2^-40) and the largest a write can set (2^119): every
    page counts in the softmax's sum, with scores alike or those of the large pages lower by 40."""
    _far_apart(h3, new, length, order, gap, 4.0)


@pytest.mark.parametrize("order", ["turn by turn", "small ones first", "large ones first"])
@pytest.mark.parametrize("new,length", [(1, 300), (9, 300), (140, 300), (1, 9_000), (20, 4_000), (140, 2_500)])
def test_large_values_of_small_probability(h3, new, length, order):
    """... or lower by 92: probabilities below FP32's smallest normal number whose values are large enough to be all of
    the output, also where they lie in a part of the keys of their own."""
    _far_apart(h3, new, length, order, 92, 12.0)


def _far_apart(h3, new, length, order, gap, q0):
    rng = np.random.default_rng(25)
    page, dim = 32, 128
    lengths = [length, 70]
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, 2, page, dim)
    c.k_scale.fill_(0.25)
    n = table.shape[1]
    large = {"turn by turn": np.arange(n) % 2 == 1, "small ones first": np.arange(n) >= n // 2,
             "large ones first": np.arange(n) < n // 2}[order]
    q = torch.randn(2 * new, 4, dim, generator=torch.Generator().manual_seed(9)).abs().mul(0.5).bfloat16().cuda()
    q[:, :, 0] = q0
    lower = -gap / (q0 * dim ** -0.5)                       # channel 0 carries the gap
    for b, most in enumerate(lengths):
        for i in range(-(-most // page)):
            p = int(table[b, i])
            c.v_scale[p] = 2.0 ** (119 if large[i] else -40)
            used = c.k_codes[p, :, :min(page, most - i * page), 0]
            used.fill_(int(O.e4m3_encode(lower * 4)) if large[i] else 0)
    cu = [0, new, 2 * new]
    out, lse = _run(h3, q, c, table, lengths, cu, new, causal=True)
    _check(h3, q, c, table, lengths, cu, out, lse, causal=True)
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("value", [0, 0x7E])
@pytest.mark.parametrize("drop", [25.1, 28.0, 31.0])
@pytest.mark.parametrize("new,heads,length", [(1, 2, 262_143), (1, 2, 700), (16, 2, 37_810), (140, 2, 37_810), (140, 80, 3_000)])
def test_many_keys_far_below_one(h3, new, heads, length, drop, value, first):
    """One key stands 2^drop above all others, which together still count (alone, where its own value is 0).

    Bound: 2^-8 of the result for its rounding, 2^-10 + 4 e of the mean of |v| as elsewhere, and for weights below FP16's
    normal numbers half a step each: 2^-25 in units in which the largest weight is 2^15 (few rows) or 2^7 at least (many),
    times the largest code, 448, of its page.  All other values are positive, so that what is lost shows."""
    rng = np.random.default_rng(26)
    page, dim = 128, 128
    n = -(-length // page)
    c = h3.KVCache.empty(n, page, heads, dim)
    k, v = np.zeros((n, heads, page, dim), dtype=np.uint8), rng.integers(0x68, 0x7F, (n, heads, page, dim)).astype(np.uint8)
    at = 0 if first else length - 1
    k[at // page, :, at % page, 0] = O.e4m3_encode(8.0)
    v[at // page, :, at % page] = value
    scale = np.float32(drop * np.log(2) / 32)                   # q . k = 32 scale: 2^drop
    c.k_codes.copy_(_dev(k, torch.uint8))
    c.v_codes.copy_(_dev(v, torch.uint8))
    c.k_scale.fill_(float(scale))
    c.v_scale.fill_(0.125)
    q = torch.zeros(new, heads, dim, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 4.0
    table = np.arange(n, dtype=np.int32)[None]
    out, lse = _run(h3, q, c, table, [length], [0, new], new, scale=1.0)
    w = np.full(length, np.exp(-32.0 * float(scale)))
    w[at] = 1.0
    e = 2.0 ** -17 * 32.0 * float(scale)
    lift = 15 if new <= 32 else 7
    for h in (0, heads - 1):
        vv = O.TABLE[v[:, h].reshape(-1, dim)[:length]] * 0.125
        ref = w @ vv / w.sum()
        tol = 2.0 ** -8 * ref + (2.0 ** -10 + 4 * e) * ref + length * 2.0 ** (-25 - lift) * 56 / w.sum()
        got = out[:, h].double().cpu().numpy()
        assert (np.abs(got - ref) <= tol).all(), (h, float((np.abs(got - ref) / tol).max()))
        want = 32.0 * float(scale) + np.log(w.sum())
        assert (np.abs(lse[:, h].double().cpu().numpy() - want) <= e + 2.0 ** -20 * (1 + abs(want))).all()


@pytest.mark.parametrize("new", [1, 140])
@pytest.mark.parametrize("size", [1.0, 1e4, 1e6, 3e7, 1e8, 3e9, 1e12, 1e20])
def test_scores_of_every_size_stay_in_range(h3, new, size):
    """Scores up to 1e21, growing along the keys and falling: no weight leaves FP16's range, the largest one wins."""
    rng = np.random.default_rng(27)
    lengths, page = [700, 333], 32
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, 2, page, 64)
    cu = [0, new, 2 * new]
    q = torch.randn(2 * new, 4, 64, generator=torch.Generator().manual_seed(9)).mul(size).bfloat16().cuda()
    out, lse = _run(h3, q, c, table, lengths, cu, new, causal=True)
    _check(h3, q, c, table, lengths, cu, out, lse, causal=True)


@pytest.mark.parametrize("new", [1, 16, 140])
@pytest.mark.parametrize("rise", [1.0, 4.9, 7.9, 8.1, 14.9, 15.1, 40.0])
def test_scores_rising_along_the_keys(h3, new, rise):
    """Each 128 keys stand 2^rise / 8 above those before, and the last ones 2^rise above the first: references that are
    held and ones that move."""
    rng = np.random.default_rng(28)
    length, page, dim = 1_100, 16, 64
    n = -(-length // page)
    table = np.arange(n, dtype=np.int32)[None]
    c = _filled(h3, rng, table, [length], n, 2, page, dim, spread=1)
    steps = np.minimum(np.arange(n) * page // 128, 8)
    k = np.zeros((n, 2, page, dim), dtype=np.uint8)
    k[..., 0] = O.e4m3_encode(steps.astype(float))[:, None, None]
    c.k_codes.copy_(_dev(k, torch.uint8))
    c.k_scale.fill_(float(np.float32(rise * np.log(2) / 8)))
    q = torch.zeros(new, 4, dim, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    out, lse = _run(h3, q, c, table, [length], [0, new], new, scale=1.0)
    _check(h3, q, c, table, [length], [0, new], out, lse, scale=1.0)


@pytest.mark.parametrize("new", [1, 20, 140])
@pytest.mark.parametrize("log_v_scale", [-40, -7, 0, 30, 100])
@pytest.mark.parametrize("window", [1, 2, 64, 0])
def test_logarithm_of_plain_counts(h3, new, log_v_scale, window):
    """With a softmax scale of 0 the log-sum-exp is the logarithm of the number of keys seen, whatever the values' scales:
    2^-21 for its rounding, and as much again for that of a base-2 logarithm below 12 (2^-22 of a part in [0, 1), the
    sum's own roundings 2^-24 each along at most four joins)."""
    rng = np.random.default_rng(29)
    lengths, page = [1_500, 260], 64
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, 2, page, 64)
    c.v_scale.fill_(2.0 ** log_v_scale)
    cu = [0, new, 2 * new]
    q = torch.randn(2 * new, 4, 64, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    out, lse = _run(h3, q, c, table, lengths, cu, new, scale=0.0, causal=True, window=window)
    _check(h3, q, c, table, lengths, cu, out, lse, scale=0.0, causal=True, window=window)
    for b, n in enumerate(lengths):
        seen = np.minimum(np.arange(n - new, n) + 1, window if window else n)
        want = np.log(seen)[:, None]
        got = lse[cu[b]:cu[b + 1]].double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -21 * np.maximum(np.abs(want), 1) + 2.0 ** -21).all(), float(np.abs(got - want).max())
