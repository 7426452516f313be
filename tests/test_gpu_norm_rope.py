"""Per-head norms of queries and keys with their rotation, and the gradients,
against the 64-bit definitions.

Forward, per value: the rounding to bf16 (2^-8 of it at most), and in FP32 a
sum of up to 256 squares (13 roundings in a row, halved by the root: 2^-21), the
root's 2 ulp (2^-22), the rotation (2^-20 of the pair, as for the rotation
alone) and three products: below 2^-19 of the pair's |a| + |b|.
Backward: g as the rotation, 2^-20 of its pair; r and the mean as above; so dx
is 2^-8 of itself and 2^-18 of the sum of magnitudes that it is made of.  dw: the
same 2^-18 of its sum of magnitudes, and 2^-24 for each addition in a row, of
which there are no more than half the rows (two groups of lanes at least share a
token's heads, or the tokens) and 100 where the lanes' sums are joined.
"""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_cache import _patterns

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _values(t):
    return O.bf16_values(_patterns(t))


def _normal(shape, seed, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).mul(scale).bfloat16().cuda()


def _weight(dim, wide, seed):
    w = 1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(seed))
    return (w if wide else w.bfloat16()).cuda()


def _rope(h3, tokens, dims, layout, seed, far=300.0):
    if dims is None:
        return None
    pos = (torch.rand(tokens, len(dims), generator=torch.Generator().manual_seed(seed)) * far).floor().cuda()
    return h3.Rope(pos, h3.rope_frequencies(dims), dims, layout=layout)


def _turn(rope, inverse=False):
    if rope is None:
        return lambda z: (z, np.abs(z))
    return lambda z: O.rope(z, rope.positions.cpu().numpy(), rope.freqs.cpu().numpy(), rope.dims, rope.layout, inverse)


def _near(got, ref, mag, units, what):
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + units * mag + 1e-38)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - ref)[bad].max()))


def _check_forward(x, w, rope, got, eps=EPS):
    ref, mag = O.norm_rope(_values(x), 1.0 if w is None else w.double().cpu().numpy(), eps, _turn(rope))
    _near(_values(got), ref, mag, 2.0 ** -19, "out")


def _check_backward(g, x, w, rope, dx, dw, eps=EPS):
    dx_ref, dw_ref, dx_mag, dw_mag = O.norm_rope_backward(_values(g), _values(x), 1.0 if w is None else w.double().cpu().numpy(),
                                                          eps, _turn(rope, inverse=True))
    _near(_values(dx), dx_ref, dx_mag, 2.0 ** -18, "dx")
    if w is None:
        assert dw is None
        return
    rows = x.shape[0] * x.shape[1]
    off = np.abs(dw.double().cpu().numpy() - dw_ref)
    assert (off <= (2.0 ** -18 + (rows / 2 + 100) * 2.0 ** -24) * dw_mag + 1e-38).all(), float((off / dw_mag).max())


CASES = [   # tokens, query heads, key heads, dim, rotated channels, layout, weights (None, bf16, FP32), extra heads in a row
    (1, 1, 1, 128, (128,), "halves", 0, 0),
    (1, 64, 8, 128, (128,), "halves", 0, 8),
    (5, 56, 56, 128, (44, 42, 42), "interleaved", 1, 56),
    (3, 2, 0, 128, (32, 48, 48), "interleaved", 0, 0),
    (37, 7, 3, 64, (16, 24, 24), "halves", 1, 1),
    (130, 5, 1, 64, (10, 12), "interleaved", None, 0),       # channels past the axes; no weight
    (6, 9, 4, 256, (64, 64, 64, 64), "halves", 0, 0),
    (9, 3, 3, 8, (2, 2, 2, 2), "interleaved", 1, 0),
    (11, 4, 2, 80, (20, 30, 30), "halves", 0, 2),            # ten lanes a head
    (7, 5, 2, 24, (0, 6, 8), "halves", 0, 0),
    (4, 3, 5, 200, (100,), "halves", 1, 0),
    (1_003, 3, 1, 96, (96,), "interleaved", 1, 1),
    (50, 6, 2, 128, None, "interleaved", 0, 0),              # no rotation
    (2_001, 2, 1, 128, (44, 42, 42), "halves", 0, 0),
    (33, 6, 3, 256, (256,), "halves", 1, 0),
    (33, 6, 3, 80, (80,), "halves", 0, 0),                   # halves that face each other across lanes that idle
    (33, 6, 3, 72, (72,), "halves", 0, 0),                   # an odd number of chunks
    (70, 9, 2, 64, (64,), "halves", 0, 0),
    (65, 3, 2, 16, (16,), "halves", 0, 0),
    (1_999, 7, 3, 256, (120, 100), "interleaved", 1, 0),
    (301, 11, 5, 40, (16, 8, 8, 8), "halves", 1, 0),
    (33, 6, 3, 128, (32, 48, 48), "halves", 0, 0),           # sections of whole chunks
    (33, 6, 3, 72, (32, 16), "halves", 1, 0),                # and channels that do not turn, an odd number of chunks
    (33, 6, 3, 256, (64, 0, 96, 16), "halves", 0, 0),
    (5, 3, 1, 8, (8,), "halves", 0, 0),
]


@pytest.mark.parametrize("tokens,hq,hk,dim,dims,layout,wide,extra", CASES)
def test_forward_and_backward_against_64_bits(h3, tokens, hq, hk, dim, dims, layout, wide, extra):
    rows = _normal((tokens, hq + hk + extra, dim), tokens + hq, 1.5)
    q, k = rows[:, :hq], rows[:, hq:hq + hk] if hk else None
    wq, wk = [None if wide is None else _weight(dim, wide, i) for i in (1, 2)]
    wk = wk if hk else None
    rope = _rope(h3, tokens, dims, layout, 3)
    before = rows.clone()
    q_out, k_out = h3.norm_rope(q, k, q_weight=wq, k_weight=wk, rope=rope, eps=EPS)
    gq, gk = _normal(q.shape, 5, 0.1), _normal(k.shape, 6, 0.1) if hk else None
    dq, dk, dwq, dwk = h3.norm_rope_backward(gq, gk, q, k, q_weight=wq, k_weight=wk, rope=rope, eps=EPS)
    assert torch.equal(rows.view(torch.int16), before.view(torch.int16))
    _check_forward(q, wq, rope, q_out)
    _check_backward(gq, q, wq, rope, dq, dwq)
    if hk:
        _check_forward(k, wk, rope, k_out)
        _check_backward(gk, k, wk, rope, dk, dwk)
    else:
        assert k_out is None and dk is None and dwk is None


def test_gradients_against_differences(h3):
    """d/dx and d/dw of sum(c * norm_rope(x)) by central differences of the 64-bit forward form.  The differences' own error
    is step^2 times a third derivative: below 1e-6 of the row's size here."""
    dims, dim, tokens, heads = (6, 10), 16, 2, 2
    rope = _rope(h3, tokens, dims, "halves", 3)
    x, c, w = _normal((tokens, heads, dim), 1), _normal((tokens, heads, dim), 2), _weight(dim, 1, 4)
    dq, _, dw, _ = h3.norm_rope_backward(c, None, x, q_weight=w, rope=rope, eps=1e-2)
    xv, cv, wv = _values(x), _values(c), w.double().cpu().numpy()

    def loss(xx, ww):
        return (cv * O.norm_rope(xx, ww, 1e-2, _turn(rope))[0]).sum()

    step = 1e-4
    got, size = _values(dq), np.abs(cv).max() * np.abs(wv).max() * 4
    for t in range(tokens):
        for h in range(heads):
            for i in range(dim):
                d = np.zeros_like(xv)
                d[t, h, i] = step
                diff = (loss(xv + d, wv) - loss(xv - d, wv)) / (2 * step)
                assert abs(diff - got[t, h, i]) <= 2.0 ** -8 * 1.01 * abs(diff) + 1e-5 * size
    for i in range(dim):
        d = np.zeros_like(wv)
        d[i] = step
        diff = (loss(xv, wv + d) - loss(xv, wv - d)) / (2 * step)
        assert abs(diff - dw[i].item()) <= 1e-5 * size * tokens * heads


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 7), (3, 5), (517, 3), (40, 56), (5_000, 2)])
def test_weight_gradients_are_whole_sums(h3, tokens, heads):
    """Rows of +-1 have r = 1 to the bit (eps vanishes), so that integers sum up exactly: no row is left out or counted
    twice, for any split."""
    g = torch.Generator().manual_seed(tokens)
    sign = torch.randint(0, 2, (tokens, heads + 2, 128), generator=g).mul(2).sub(1)
    dy = torch.randint(-8, 9, (tokens, heads + 2, 128), generator=g)
    x, d = sign.bfloat16().cuda(), dy.bfloat16().cuda()
    one = torch.ones(128, device="cuda")
    _, _, dwq, dwk = h3.norm_rope_backward(d[:, :heads], d[:, heads:], x[:, :heads], x[:, heads:], q_weight=one, k_weight=one,
                                           eps=2.0 ** -100)
    want = (sign * dy).double()
    assert torch.equal(dwq.double().cpu(), want[:, :heads].sum((0, 1)))
    assert torch.equal(dwk.double().cpu(), want[:, heads:].sum((0, 1)))


def test_rows_of_any_size(h3):
    """Rows whose squares leave FP32's range, zero rows, tiny ones, and rows with infinities and NaN, side by side."""
    sizes = torch.tensor([1.0, 0.0, 1e-30, 3e38, 1e25, 2.0 ** 60, 2.0 ** 50, 1e-3], device="cuda")
    x = (_normal((3, 8, 128), 7).clamp(-0.99, 0.99).float() * sizes[None, :, None]).bfloat16()
    w = _weight(128, 1, 1)
    rope = _rope(h3, 3, (44, 42, 42), "interleaved", 2)
    _check_forward(x, w, rope, h3.norm_rope(x, q_weight=w, rope=rope)[0])
    g = _normal(x.shape, 8)
    dq, _, dw, _ = h3.norm_rope_backward(g, None, x, q_weight=w, rope=rope)
    _check_backward(g, x, w, rope, dq, dw)
    clean = h3.norm_rope(x, q_weight=w, rope=rope)[0]
    x[1, 0, 3], x[1, 7, 100] = float("inf"), float("nan")
    y = h3.norm_rope(x, q_weight=w, rope=rope)[0]
    assert y[1, 7].isnan().all() and y[1, 0, 2:4].isnan().all()      # (an infinity's pair)
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[2:4] = False
    assert (y[1, 0, rest] == 0).all()
    keep = torch.ones(3, 8, dtype=torch.bool, device="cuda")
    keep[1, 0] = keep[1, 7] = False
    assert torch.equal(y[keep].view(torch.int16), clean[keep].view(torch.int16))


@pytest.mark.parametrize("layout,dims,still,turned,pair", [("interleaved", (10, 16), 27, 5, 4), ("halves", (10, 16), 27, 5, 0),
                                                           ("halves", (16, 16), 45, 21, 29)])
def test_an_infinity_stays_in_its_pair_beside_channels_that_do_not_turn(h3, layout, dims, still, turned, pair):
    x = _normal((2, 2, 64), 7)
    x[0, 0, still], x[1, 1, turned] = float("inf"), float("-inf")
    rope = _rope(h3, 2, dims, layout, 2)
    y = h3.norm_rope(x, rope=rope)[0]
    assert y[0, 0, still].isnan() and y[1, 1, turned].isnan() and y[1, 1, pair].isnan()
    assert int(y[0, 0].isnan().sum()) == 1 and int(y[1, 1].isnan().sum()) == 2
    assert (y[0, 0][~y[0, 0].isnan()] == 0).all() and y[0, 1].isfinite().all()
    g = _normal(x.shape, 8)
    g[0, 1, 47] = float("inf")
    one = torch.ones(64, device="cuda")
    _, _, dw, _ = h3.norm_rope_backward(g, None, _normal(x.shape, 9), q_weight=one, rope=rope)
    assert not dw[47].isfinite() and int((~dw.isfinite()).sum()) == 1


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_in_place_in_the_rows_of_a_projection(h3, layout):
    """Grouped heads side by side in one projection's rows, normed in place; gradients over those of the outputs, and over x."""
    rows = _normal((67, 12, 128), 3)
    rope = _rope(h3, 67, (44, 42, 42), layout, 4)
    w = _weight(128, 0, 1), _weight(128, 0, 2)
    q, k = rows[:, :7], rows[:, 7:9]
    want = h3.norm_rope(q, k, q_weight=w[0], k_weight=w[1], rope=rope)
    grads = _normal((67, 9, 128), 5)
    gq, gk = grads[:, :7], grads[:, 7:]
    back = h3.norm_rope_backward(gq, gk, q, k, q_weight=w[0], k_weight=w[1], rope=rope)
    over_x = rows.clone()
    h3.norm_rope_backward(gq, gk, over_x[:, :7], over_x[:, 7:9], q_weight=w[0], k_weight=w[1], rope=rope, q_out=over_x[:, :7],
                          k_out=over_x[:, 7:9])
    assert torch.equal(over_x[:, :7], back[0]) and torch.equal(over_x[:, 7:9], back[1]) and torch.equal(over_x[:, 9:], rows[:, 9:])
    got = h3.norm_rope_backward(gq, gk, q, k, q_weight=w[0], k_weight=w[1], rope=rope, q_out=gq, k_out=gk)
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    rest = rows[:, 9:].clone()
    h3.norm_rope(q, k, q_weight=w[0], k_weight=w[1], rope=rope, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(rows[:, 9:], rest)


def test_streams_repeats_and_graphs(h3):
    """The same bits on another stream, in repeats and from a replayed graph whose inputs changed."""
    x = _normal((1_500, 9, 64), 1)
    g = _normal(x.shape, 2)
    w = _weight(64, 1, 3)
    rope = _rope(h3, 1_500, (64,), "halves", 4)

    def both(stream=None):
        y = h3.norm_rope(x[:, :6], x[:, 6:], q_weight=w, k_weight=w, rope=rope, stream=stream)
        return y + h3.norm_rope_backward(g[:, :6], g[:, 6:], x[:, :6], x[:, 6:], q_weight=w, k_weight=w, rope=rope, stream=stream)

    want = both()
    assert all(torch.equal(a, b) for _ in range(3) for a, b in zip(both(), want))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = both(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = both()
    for seed in (5, 6):
        x.copy_(_normal(x.shape, seed))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_nothing_to_do(h3):
    w = _weight(128, 1, 1)
    x = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    rope = _rope(h3, 0, (128,), "halves", 1)
    assert h3.norm_rope(x, x[:, :2], q_weight=w, k_weight=w, rope=rope)[1].shape == (0, 2, 128)
    full = torch.full((128,), 7.0, device="cuda")
    _, _, dw, none = h3.norm_rope_backward(x, None, x, q_weight=w, rope=rope, q_weight_grad=full)
    assert none is None and dw is full and (dw == 0).all()
    rows = _normal((4, 3, 128), 2)
    no_heads = rows[:, :0]
    _, dk, dwq, dwk = h3.norm_rope_backward(no_heads, rows, no_heads, rows, q_weight=w, k_weight=w)
    assert (dwq == 0).all() and (dwk != 0).any() and dk.shape == rows.shape


def test_offsets_past_32_bits(h3):
    tokens = 4_400_000
    wide = torch.empty(tokens, 8, 128, dtype=torch.bfloat16, device="cuda")
    tail = _normal((5, 8, 128), 1)
    wide[-5:] = tail
    wide[:-5, :1] = 1
    w = _weight(128, 0, 1)
    pos = torch.zeros(tokens, 1, device="cuda")
    pos[-5:] = 9.0
    freqs = h3.rope_frequencies((128,))
    h3.norm_rope(wide[:, :1], q_weight=w, rope=h3.Rope(pos, freqs, (128,)), q_out=wide[:, :1])
    want = h3.norm_rope(tail[:, :1], q_weight=w, rope=h3.Rope(pos[-5:], freqs, (128,)))[0]
    assert torch.equal(wide[-5:, :1], want) and torch.equal(wide[-5:, 1:], tail[:, 1:])


@pytest.mark.parametrize("tokens,hq,hk,dim,dims,wide", [
    (5, 4, 3, 256, (88, 84, 84), 0),            # sections that are not whole chunks, over all of the widest head
    (7, 5, 2, 256, (10, 246), 1),
    (6, 7, 4, 256, (10, 30, 208), 0),
    (9, 3, 0, 256, (120,), 0),                  # and over a part of it
    (8, 9, 5, 256, (254,), None),
    (4, 6, 3, 248, (248,), 1),
    (5, 3, 4, 248, (82, 82, 84), 0),
    (61, 11, 7, 240, (120, 120), 0),
    (5, 5, 3, 136, (12, 124), 1),
    (9, 13, 5, 128, (10, 118), 0),              # the widest of eight lanes, and of four
    (9, 17, 9, 64, (10, 54), 1),
    (700, 8, 3, 256, (88, 84, 84), 1),
])
def test_widest_heads_in_halves_of_uneven_sections(h3, tokens, hq, hk, dim, dims, wide):
    """Forward and backward, then in place in a projection's rows: each head of a warp keeps its own words while they are
    exchanged."""
    rows, rope = _normal((tokens, hq + hk + 1, dim), tokens + hq, 1.5), _rope(h3, tokens, dims, "halves", 3)
    q, k = rows[:, :hq], rows[:, hq:hq + hk] if hk else None
    wq, wk = [None if wide is None else _weight(dim, wide, i) for i in (1, 2)]
    wk = wk if hk else None
    gq, gk = _normal(q.shape, 5, 0.1), _normal(k.shape, 6, 0.1) if hk else None
    kw = dict(q_weight=wq, k_weight=wk, rope=rope, eps=EPS)
    out, back = h3.norm_rope(q, k, **kw), h3.norm_rope_backward(gq, gk, q, k, **kw)
    for x, w, y, g, dx, dw in ((q, wq, out[0], gq, back[0], back[2]), (k, wk, out[1], gk, back[1], back[3])):
        if x is not None:
            _check_forward(x, w, rope, y)
            _check_backward(g, x, w, rope, dx, dw)
    over = h3.norm_rope_backward(gq, gk, q, k, q_out=gq, k_out=gk, **kw)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(over, back))
    h3.norm_rope(q, k, q_out=q, k_out=k, **kw)
    assert torch.equal(q, out[0]) and (k is None or torch.equal(k, out[1]))
