"""Rotary positions with several axes against the 64-bit definition.

Bound per value: the rounding to bf16, 2^-8 of the result (half an ulp is at
most 2^-8 of the value), plus the FP32 rotation.  The reduced angle is below
half a turn and carries at most 2^-26 turns of rounding (2 pi 2^-26 < 2^-23
radians) plus 2^-48 of the unreduced angle in turns; sincospi adds 2 ulp
(2^-23) and the two products and the sum 2^-24 each: below 2^-20 (|a| + |b|)
for angles up to 2^24 turns, with a factor of four to spare.
"""
import numpy as np
import pytest
import torch

from oracle import attention as O

pytestmark = pytest.mark.gpu


def _check(y, ref, mag):
    got = O.bf16_values(y.cpu().view(torch.int16).numpy().view(np.uint16))
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + 2.0 ** -20 * mag + 1e-38
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref)[bad].max()))


def _inputs(tokens, heads, dim, dims, seed, extra_heads=0, far=200.0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(tokens, heads + extra_heads, dim, generator=g).to(torch.bfloat16).cuda()
    pos = (torch.rand(tokens, len(dims), generator=g) * far).floor().cuda()
    return wide, pos


CASES = [
    (1, 1, 128, (44, 42, 42), "interleaved", 0),
    (1, 112, 128, (44, 42, 42), "halves", 0),
    (5, 56, 128, (32, 48, 48), "interleaved", 56),
    (37, 7, 64, (16, 24, 24), "halves", 3),
    (9, 3, 64, (10, 12), "interleaved", 0),          # channels past the axes are copied
    (130, 5, 128, (128,), "halves", 1),
    (6, 9, 256, (64, 64, 64, 64), "halves", 0),
    (6, 9, 8, (2, 2, 2, 2), "interleaved", 0),
    (11, 4, 80, (20, 30, 30), "halves", 2),          # ten lanes a head: three heads a warp, two lanes idle
    (3, 2, 24, (0, 6, 8), "halves", 0),              # an axis without channels
    (4, 2, 16, (0,), "interleaved", 0),              # nothing turns
]


@pytest.mark.parametrize("tokens,heads,dim,dims,layout,extra", CASES)
def test_forward_and_inverse_against_64_bits(h3, tokens, heads, dim, dims, layout, extra):
    wide, pos = _inputs(tokens, heads, dim, dims, tokens + heads, extra)
    x = wide[:, :heads]
    freqs = h3.rope_frequencies(dims)
    r = h3.Rope(pos, freqs, dims, layout=layout)
    before = wide.clone()
    xv = O.bf16_values(x.cpu().contiguous().view(torch.int16).numpy().view(np.uint16))
    for inverse in (False, True):
        ref, mag = O.rope(xv, pos.cpu().numpy(), freqs.cpu().numpy(), dims, layout, inverse)
        _check(h3.rope_axes(x, r, inverse=inverse), ref, mag)
    assert torch.equal(wide.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_in_place_and_strided_output_give_the_same_bits(h3, layout):
    dims = (44, 42, 42)
    wide, pos = _inputs(67, 12, 128, dims, 5, 12)
    r = h3.Rope(pos, h3.rope_frequencies(dims), dims, layout=layout)
    want = h3.rope_axes(wide[:, :12], r)
    out = torch.full((12, 67, 128), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)   # heads outermost
    h3.rope_axes(wide[:, :12], r, out=out)
    assert torch.equal(out, want)
    rest = wide[:, 12:].clone()
    h3.rope_axes(wide[:, :12], r, out=wide[:, :12])
    assert torch.equal(wide[:, :12], want) and torch.equal(wide[:, 12:], rest)


def test_inverse_is_the_gradient(h3):
    """d/dx of sum(w * rope(x)) by central differences of the 64-bit forward map, against the inverse applied to w."""
    dims = (6, 10)
    wide, pos = _inputs(3, 2, 16, dims, 8)
    freqs = h3.rope_frequencies(dims)
    r = h3.Rope(pos, freqs, dims, layout="halves")
    w = torch.randn(3, 2, 16, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    grad = O.bf16_values(h3.rope_axes(w, r, inverse=True).cpu().view(torch.int16).numpy().view(np.uint16))
    xv = wide.cpu().double().numpy()
    wv, p, f = w.cpu().double().numpy(), pos.cpu().numpy(), freqs.cpu().numpy()
    for t in range(3):
        for c in range(16):
            d = np.zeros_like(xv)
            d[t, 1, c] = 0.5
            diff = (wv * (O.rope(xv + d, p, f, dims, "halves")[0] - O.rope(xv - d, p, f, dims, "halves")[0])).sum()
            assert abs(diff - grad[t, 1, c]) <= 2.0 ** -8 * 1.01 * abs(diff) + 2.0 ** -18 * np.abs(wv[t, 1]).max()


def test_far_and_fractional_positions(h3):
    """Positions up to 2^23 and fractions: the reduction keeps the angle exact."""
    dims = (64,)
    wide, _ = _inputs(8, 2, 64, dims, 9)
    pos = torch.tensor([[0.0], [0.5], [-3.25], [131_071.0], [1_000_003.0], [8_388_607.0], [-8_388_606.0], [77_777.75]],
                       device="cuda")
    freqs = h3.rope_frequencies(dims)
    r = h3.Rope(pos, freqs, dims)
    xv = wide.cpu().double().numpy()
    ref, mag = O.rope(xv, pos.cpu().numpy(), freqs.cpu().numpy(), dims, "interleaved")
    _check(h3.rope_axes(wide, r), ref, mag)


def test_special_values(h3):
    """Channels that do not turn are copied bit for bit, infinities and NaN stay with their pair."""
    x = torch.randn(1, 1, 16, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    x[0, 0, 0], x[0, 0, 9], x[0, 0, 12] = float("nan"), float("inf"), -0.0
    r = h3.Rope(torch.tensor([[3.0]], device="cuda"), h3.rope_frequencies((8,)), (8,))
    y = h3.rope_axes(x, r)
    assert torch.equal(y[0, 0, 8:].view(torch.int16), x[0, 0, 8:].view(torch.int16))
    assert y[0, 0, :2].isnan().all() and y[0, 0, 2:8].isfinite().all()


def test_another_stream_and_no_tokens(h3):
    dims = (32, 48, 48)
    wide, pos = _inputs(513, 4, 128, dims, 12)
    r = h3.Rope(pos, h3.rope_frequencies(dims), dims)
    want = h3.rope_axes(wide, r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(wide)
    h3.rope_axes(wide, r, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    assert h3.rope_axes(wide[:0], r).shape == (0, 4, 128)


def test_offsets_past_32_bits(h3):
    """Rows whose byte and element offsets pass 2^32: the last rows of a 4.5e9-element array of which few are used."""
    dims = (32, 48, 48)
    tokens, ld = 4_400_000, 8 * 128
    wide = torch.empty(tokens, 8, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    tail = torch.randn(5, 8, 128, generator=g, device="cuda").bfloat16()
    wide[-5:] = tail
    pos = torch.zeros(tokens, 3, device="cuda")
    pos[-5:] = torch.tensor([3.0, 5.0, 7.0], device="cuda")
    r = h3.Rope(pos, h3.rope_frequencies(dims), dims)
    assert tokens * ld > 2 ** 32
    h3.rope_axes(wide[:, :1], r, out=wide[:, :1])
    want = h3.rope_axes(tail[:, :1], h3.Rope(pos[-5:], r.freqs, dims))
    assert torch.equal(wide[-5:, :1], want) and torch.equal(wide[-5:, 1:], tail[:, 1:])


@pytest.mark.parametrize("heads,dim,dims,layout", [(3, 128, (44, 42, 42), "halves"), (1, 80, (20, 30, 30), "halves"), (5, 64, (16, 24, 24), "halves"),
                                                   (2, 256, (64, 64, 64, 64), "halves"), (3, 128, (32, 48, 48), "interleaved")])
def test_many_tokens_give_the_bits_of_few(h3, heads, dim, dims, layout):
    """A long call (5,003 tokens) against the definition, and against its own tokens in calls of a few."""
    wide, pos = _inputs(5_003, heads, dim, dims, 9, 1)
    x, freqs = wide[:, 1:], h3.rope_frequencies(dims)
    y = h3.rope_axes(x, h3.Rope(pos, freqs, dims, layout=layout))
    xv = O.bf16_values(x.cpu().contiguous().view(torch.int16).numpy().view(np.uint16))
    ref, mag = O.rope(xv, pos.cpu().numpy(), freqs.cpu().numpy(), dims, layout, False)
    _check(y, ref, mag)
    for at, n in ((0, 13), (2_431, 20), (4_996, 7)):
        part = h3.rope_axes(x[at:at + n], h3.Rope(pos[at:at + n].contiguous(), freqs, dims, layout=layout))
        assert torch.equal(part.view(torch.int16), y[at:at + n].view(torch.int16))
