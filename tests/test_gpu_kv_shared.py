"""Attention of sequences that share prefixes, against the 64-bit definition on
each sequence's prefix and own keys side by side.  Bounds as for the attention
over one cache: the join of two halves adds a few FP32 roundings, for which the
2^-10 of the weighted mean leaves room."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_attention import _filled
from test_gpu_kv_cache import _dev, _patterns, _tables
from test_gpu_kv_sinks import check_rows

pytestmark = pytest.mark.gpu


def _setup(h3, seed, groups, seqs, heads, kv_heads, dim, page):
    """groups: (prefix length, sequences); seqs: (new, own keys) of each sequence."""
    rng = np.random.default_rng(seed)
    lengths = [L for _, L in seqs] + [p for p, _ in groups]
    table, pages = _tables(rng, lengths, page)
    c = _filled(h3, rng, table, lengths, pages, kv_heads, page, dim)
    new = [n for n, _ in seqs]
    cu = np.cumsum([0] + new)
    first = np.cumsum([0] + [n for _, n in groups])
    p_cu = cu[first]
    q = torch.randn(cu[-1] + 3, heads, dim, generator=torch.Generator().manual_seed(seed)).mul(2).bfloat16().cuda()
    return c, q, table[:len(seqs)], table[len(seqs):], cu, p_cu, first


def _call(h3, c, q, own, shared, groups, seqs, cu, p_cu, **kw):
    prefix = h3.SharedPrefix(_dev(shared), _dev([p for p, _ in groups]), _dev(p_cu), int(np.diff(p_cu).max(initial=0)),
                             max([p for p, _ in groups], default=0))
    return h3.kv_attention_shared(q, c, prefix, _dev(own), _dev([L for _, L in seqs]), _dev(cu), max(n for n, _ in seqs),
                                  max(L for _, L in seqs), return_lse=True, **kw)


def _check(c, q, own, shared, groups, seqs, cu, first, out, lse, causal, scale=None):
    kv, vv = [O.cache_values(t.cpu().numpy(), s.cpu().numpy()) for t, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))]
    qv, got, gl = O.bf16_values(_patterns(q)), O.bf16_values(_patterns(out)), lse.cpu().numpy()
    for b, (n, L) in enumerate(seqs):
        g = [i for i in range(len(groups)) if first[i] <= b < first[i + 1]]
        P = groups[g[0]][0] if g else 0
        k, v = [np.concatenate([O.gather(x, shared[g[0]], P), O.gather(x, own[b], L)]) if g else O.gather(x, own[b], L) for x in (kv, vv)]
        at = slice(int(cu[b]), int(cu[b + 1]))
        check_rows(qv[at], k, v, got[at], gl[at], q.shape[2] ** -0.5 if scale is None else scale, P + L, causal=causal, before=P)


CASES = [   # (prefix, sequences) of each group, (new, own keys) of each sequence, heads, kv_heads, dim, page, causal
    ([(1, 1)], [(1, 1)], 1, 1, 128, 16, 1),
    ([(777, 3)], [(1, 40), (1, 1), (1, 17)], 16, 4, 64, 16, 1),
    ([(300, 2), (65, 3)], [(1, 5), (1, 33), (1, 200), (1, 64), (1, 1)], 8, 2, 128, 64, 1),
    ([(500, 4)], [(1, 2000), (1, 0), (1, 3), (1, 900)], 8, 8, 128, 32, 0),     # own keys: none, and more than the prefix
    ([(0, 1), (90, 1)], [(2, 7), (3, 9)], 4, 2, 64, 16, 1),                    # an empty prefix
    ([(90, 0), (33, 2)], [(2, 7), (3, 2)], 4, 4, 128, 16, 1),                  # an empty group; more queries than own keys
    ([(2000, 40)], [(1, 3 + 11 * i) for i in range(40)], 8, 1, 128, 64, 1),    # many rows over the prefix, few over own keys
    ([(130, 2)], [(70, 80), (129, 129)], 4, 2, 128, 16, 1),                    # many over both
    ([(1300, 3), (40, 1)], [(70, 70), (1, 90), (30, 30), (257, 300)], 2, 2, 64, 128, 0),
    ([(513, 2)], [(5, 6), (0, 0)], 6, 3, 128, 128, 1),                         # a sequence without tokens
    ([(3000, 1)], [(1, 3000)], 5, 1, 128, 64, 0),
    ([(257, 20)], [(2, 1500)] * 20, 4, 4, 64, 32, 1),
]


@pytest.mark.parametrize("groups,seqs,heads,kv_heads,dim,page,causal", CASES)
def test_against_64_bits(h3, groups, seqs, heads, kv_heads, dim, page, causal):
    c, q, own, shared, cu, p_cu, first = _setup(h3, heads * 10 + len(seqs), groups, seqs, heads, kv_heads, dim, page)
    wide = torch.full((q.shape[0], heads + 2, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], heads), 5.0, device="cuda")
    out, _ = _call(h3, c, q, own, shared, groups, seqs, cu, p_cu, causal=bool(causal), out=wide[:, 1:1 + heads], lse=lse)
    assert h3.h3fp4_device_error() == 0
    _check(c, q, own, shared, groups, seqs, cu, first, out, lse, bool(causal))
    assert (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all() and (wide[cu[-1]:] == 7).all() and (lse[cu[-1]:] == 5).all()


@pytest.mark.parametrize("new,batch", [(1, 3), (1, 12), (40, 2)])
def test_rows_of_no_group_have_no_prefix(h3, new, batch):
    """Groups that cover the middle sequences, or none at all."""
    seqs = [(new, 60 + new * b) for b in range(batch)]
    c, q, own, shared, cu, p_cu, first = _setup(h3, batch, [(333, 1)], seqs, 8, 2, 128, 32)
    for at in ((1, 2), (1, 1)):
        out, lse = _call(h3, c, q, own, shared, [(333, 1)], seqs, cu, cu[list(at)], causal=True)
        _check(c, q, own, shared, [(333, 1)], seqs, cu, at, out, lse, True)
    none = h3.SharedPrefix(torch.empty(0, 1, dtype=torch.int32, device="cuda"), _dev(np.zeros(0)), _dev([0]), 0, 0)
    out, lse = h3.kv_attention_shared(q, c, none, _dev(own), _dev([L for _, L in seqs]), _dev(cu), new, max(L for _, L in seqs),
                                      causal=True, return_lse=True)
    want = h3.kv_attention(q, c, _dev(own), _dev([L for _, L in seqs]), _dev(cu), new, max(L for _, L in seqs), causal=True,
                           return_lse=True)
    n = int(cu[-1])
    assert torch.equal(out[:n], want[0][:n]) and torch.equal(lse[:n], want[1][:n])
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("new,batch", [(1, 3), (1, 40), (50, 3)])
def test_nan_and_far_scales_in_either_half(h3, new, batch):
    seqs, groups = [(new, 100 + b) for b in range(batch)], [(400, batch)]
    c, q, own, shared, cu, p_cu, first = _setup(h3, 5, groups, seqs, 4, 2, 128, 32)
    c.v_codes[int(shared[0, 3]), 0, 5, 9] = 0x7F                       # one channel of the first cache head, all rows
    c.v_codes[int(own[1, 1]), 1, 2, 70] = 0x7F                         # one sequence
    c.k_codes[int(own[2, 0]), 0, 2, 1] = 0x7F                          # all channels of a sequence's first head
    out, lse = _call(h3, c, q, own, shared, groups, seqs, cu, p_cu)
    _check(c, q, own, shared, groups, seqs, cu, first, out, lse, False)
    for first_scale, rest in ((-40, 60), (60, -40)):
        c.v_scale.fill_(2.0 ** rest)
        c.v_scale[_dev(shared[0, :13], torch.int64)] = 2.0 ** first_scale
        out, lse = _call(h3, c, q, own, shared, groups, seqs, cu, p_cu)
        _check(c, q, own, shared, groups, seqs, cu, first, out, lse, False)


def test_halves_far_apart(h3):
    """A prefix whose scores lie far above the own keys', and far below: what is left of the other half still counts."""
    groups, seqs = [(128, 2)], [(1, 64), (60, 64)]
    c, q, own, shared, cu, p_cu, first = _setup(h3, 6, groups, seqs, 2, 2, 128, 32)
    for up in (1.0, 2.0 ** -4, 2.0 ** 4):
        c.k_scale.fill_(2.0 ** -5)
        c.k_scale[_dev(shared[0, :4], torch.int64)] = up
        out, lse = _call(h3, c, q, own, shared, groups, seqs, cu, p_cu)
        _check(c, q, own, shared, groups, seqs, cu, first, out, lse, False)


@pytest.mark.parametrize("new,batch", [(1, 4), (1, 40), (40, 3)])
def test_streams_repeats_and_graphs(h3, new, batch):
    """The same bits on two streams in turn and in repeats; a captured call follows lengths on the device."""
    seqs, groups = [(new, 300 + b) for b in range(batch)], [(700, batch)]
    c, q, own, shared, cu, p_cu, first = _setup(h3, 7, groups, seqs, 8, 2, 128, 64)
    want = _call(h3, c, q, own, shared, groups, seqs, cu, p_cu, causal=True)
    torch.cuda.synchronize()
    n, streams = int(cu[-1]), [torch.cuda.Stream() for _ in range(2)]
    kv, p_len = _dev([L for _, L in seqs]), _dev([700])
    prefix = h3.SharedPrefix(_dev(shared), p_len, _dev(p_cu), n, 700)
    args = q, c, prefix, _dev(own), kv, _dev(cu), new, 340
    torch.cuda.synchronize()
    got = [h3.kv_attention_shared(*args, causal=True, return_lse=True, stream=streams[i % 2]) for i in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o[:n], want[0][:n]) and torch.equal(l[:n], want[1][:n]) for o, l in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        out, lse = h3.kv_attention_shared(*args, causal=True, return_lse=True)
    for drop, p in ((0, 700), (100, 64), (59, 0)):
        kv.copy_(_dev([L - drop for _, L in seqs]))
        p_len.copy_(_dev([p]))
        graph.replay()
        torch.cuda.synchronize()
        _check(c, q, own, shared, [(p, batch)], [(m, L - drop) for m, L in seqs], cu, first, out, lse, True)
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("new", [1, 140])
def test_out_of_range_entries_are_reported(h3, new):
    seqs, groups = [(new, 32)], [(32, 1)]
    c, q, own, shared, cu, p_cu, first = _setup(h3, 8, groups, seqs, 2, 2, 64, 16)
    table = np.array([[0, 1]])
    for kw in (dict(shared=[[0, 99]]), dict(shared=[[-7, 1]]), dict(p=33), dict(p=-1), dict(p_cu=[0, new + 9]), dict(p_cu=[5, 0]),
               dict(own=[[0, 99]]), dict(L=33)):
        prefix = h3.SharedPrefix(_dev(kw.get("shared", table)), _dev([kw.get("p", 32)]), _dev(kw.get("p_cu", [0, new])), new, 32)
        h3.kv_attention_shared(q, c, prefix, _dev(kw.get("own", table)), _dev([kw.get("L", 32)]), _dev([0, new]), new, 32)
        assert h3.h3fp4_device_error() == 512, kw
    prefix = h3.SharedPrefix(_dev(table), _dev([32]), _dev([0, new]), new, 32)
    h3.kv_attention_shared(q, c, prefix, _dev(table), _dev([32]), _dev([0, new]), new, 32)
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("groups,seqs", [
    ([(2_000, 1)], [(1, 300), (90, 400), (64, 64)]),        # few queries over the prefix, many over own keys
    ([(300, 1), (900, 1)], [(2, 40), (1, 700), (150, 151)]),
    ([(3_000, 2)], [(150, 150), (1, 1), (3, 5_000)]),
])
def test_groups_that_cover_some_of_the_sequences(h3, groups, seqs):
    c, q, own, shared, cu, p_cu, first = _setup(h3, 21, groups, seqs, 8, 4, 128, 64)
    out, lse = _call(h3, c, q, own, shared, groups, seqs, cu, p_cu, causal=True)
    assert h3.h3fp4_device_error() == 0
    _check(c, q, own, shared, groups, seqs, cu, first, out, lse, True)


@pytest.mark.parametrize("new,batch", [(1, 3), (1, 40), (90, 2)])
def test_nothing_before_or_nothing_own(h3, new, batch):
    """Prefixes without keys, own keys without any, and both, with the largest lengths given as 0."""
    for P, L in ((0, new + 30), (200, 0), (0, 0)):
        seqs, groups = [(new, L)] * batch, [(P, batch)]
        c, q, own, shared, cu, p_cu, first = _setup(h3, 22, groups, seqs, 4, 2, 64, 16)
        out, lse = _call(h3, c, q, own, shared, groups, seqs, cu, p_cu)
        assert h3.h3fp4_device_error() == 0
        _check(c, q, own, shared, groups, seqs, cu, first, out, lse, False)


@pytest.mark.parametrize("new,batch,own,dim", [(1, 6, 40, 128), (1, 70, 90, 128), (1, 6, 3_000, 64), (1, 30, 2_000, 128), (90, 6, 120, 128),
                                               (90, 6, 120, 64), (300, 4, 700, 128), (3, 12, 50, 64)])
def test_rows_of_a_refused_group_stay_as_they_were(h3, new, batch, own, dim):
    """One group of three is out of range, in each way that its lengths and rows can be: its rows are neither written nor
    joined to anything, and the others' are right."""
    few = max(1, batch // 6)
    sizes = [few, batch - 2 * few, few]
    groups, seqs = [(200, n) for n in sizes], [(new, own + b) for b in range(batch)]
    heads = 4
    c, q, table, shared, cu, p_cu, first = _setup(h3, batch + own, groups, seqs, heads, 2, dim, 16)
    kv, vv = [O.cache_values(t.cpu().numpy(), s.cpu().numpy()) for t, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))]
    qv, most = O.bf16_values(_patterns(q)), int(np.diff(p_cu).max())
    args = _dev(table), _dev([L for _, L in seqs]), _dev(cu), new, own + batch - 1
    past = p_cu.copy()
    past[-1] = q.shape[0] + 1
    for refused, lens, rows, most_rows, most_keys in (
            (None, [200] * 3, p_cu, most, 10_000),
            (0, [-1, 200, 200], p_cu, most, 200),
            (1, [200, 201, 200], p_cu, most, 200),
            (2, [200, 200, 16 * shared.shape[1] + 1], p_cu, most, 10_000),      # past the table
            (1, [200] * 3, p_cu, most - 1, 200),                # more rows than said
            (2, [200] * 3, past, most + 9, 200)):               # rows past the arrays
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], 5.0, device="cuda")
        prefix = h3.SharedPrefix(_dev(shared), _dev(lens), _dev(rows), most_rows, most_keys)
        need = h3.h3fp4_kv_attention_shared_workspace(q.shape[0], heads, 2, dim, 3, most_rows, most_keys, batch, new, own + batch - 1)
        ws = torch.full((need,), 0x40, dtype=torch.uint8, device="cuda")        # (what scratch held: 3.0 in every place)
        h3.kv_attention_shared(q, c, prefix, *args, causal=True, out=out, lse=lse, workspace=ws)
        assert h3.h3fp4_device_error() == (0 if refused is None else 512)
        got, gl = O.bf16_values(_patterns(out)), lse.cpu().numpy()
        for b in range(batch):
            g, at = int(np.searchsorted(first, b, side="right")) - 1, slice(int(cu[b]), int(cu[b + 1]))
            if g == refused:
                assert (got[at] == 7).all() and (gl[at] == 5).all(), (refused, b)
            elif b % max(1, batch // 6) == 0:
                k, v = [np.concatenate([O.gather(x, shared[g], 200), O.gather(x, table[b], own + b)]) for x in (kv, vv)]
                check_rows(qv[at], k, v, got[at], gl[at], dim ** -0.5, 200 + own + b, causal=True, before=200)
        assert (out[cu[-1]:] == 7).all() and (lse[cu[-1]:] == 5).all()


@pytest.mark.parametrize("new,heads", [(1, 4), (40, 4), (3, 64)])
def test_groups_said_to_be_empty(h3, new, heads):
    """The most rows of a group given as 0: right where all groups are empty, and where one is not its rows are out of range."""
    groups, seqs = [(200, 1)] * 3, [(new, 50 + b) for b in range(3)]
    c, q, own, shared, cu, p_cu, first = _setup(h3, new, groups, seqs, heads, 2, 128, 32)
    args = _dev(own), _dev([L for _, L in seqs]), _dev(cu), new, 52
    want = h3.kv_attention(q, c, *args, causal=True, return_lse=True)
    n = int(cu[-1])
    for rows, refused in (([0, 0, 0, 0], None), ([n, n, n, n], None), ([0, 0, new, new], 0), (p_cu, slice(None))):
        out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], 5.0, device="cuda")
        prefix = h3.SharedPrefix(_dev(shared), _dev([200] * 3), _dev(rows), 0, 200)
        h3.kv_attention_shared(q, c, prefix, *args, causal=True, out=out, lse=lse)
        assert h3.h3fp4_device_error() == (0 if refused is None else 512)
        gone = torch.zeros(3, dtype=torch.bool)
        if refused is not None:
            gone[refused] = True
        for b in range(3):
            at = slice(b * new, b * new + new)
            if gone[b]:
                assert (out[at] == 7).all() and (lse[at] == 5).all()
            else:
                check = [[(0, 0)] * 3, [seqs[b]], cu[b:b + 2] - cu[b], [0, 0, 0, 0]]
                _check(c, q[at], own[b:b + 1], shared, *check, out[at], lse[at], True)
                assert (out[at].float() - want[0][at].float()).abs().max() <= 2.0 ** -7 * want[0][at].float().abs().max()


@pytest.mark.parametrize("new", [1, 100])
def test_halves_past_32_bits(h3, new):
    """The last rows of a call whose prefix halves take 10 GB, against the same rows in a small call."""
    groups, seqs, many = [(200, 1)], [(new, 150)], 300_000
    c, q, own, shared, cu, p_cu, first = _setup(h3, 31, groups, seqs, 64, 8, 128, 64)
    want = _call(h3, c, q[:new], own, shared, groups, seqs, cu, p_cu, causal=True)
    wide = torch.empty(many, 64, 128, dtype=torch.bfloat16, device="cuda")
    wide[-new:] = q[:new]
    at = _dev([many - new, many])
    prefix = h3.SharedPrefix(_dev(shared), _dev([200]), at, new, 200)
    out, lse = h3.kv_attention_shared(wide, c, prefix, _dev(own), _dev([150]), at, new, 150, causal=True, return_lse=True)
    assert h3.h3fp4_device_error() == 0
    assert torch.equal(out[-new:], want[0]) and torch.equal(lse[-new:], want[1])
