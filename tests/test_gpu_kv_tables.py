"""The batch's tables from its lengths, against one token after another on the
host: whole numbers, all equal."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_kv_cache import _dev

pytestmark = pytest.mark.gpu


def _inputs(rng, held, count, page, spare=3, first=0, room=1):
    held, count = np.array(held, dtype=np.int64), np.array(count, dtype=np.int64)
    begun, all_ = -(-held // page), -(-(held + count) // page)
    pages = int(all_.sum()) + spare + first
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(held), int(all_.max(initial=0)) + room), -9, dtype=np.int32)
    at = 0
    for b, n in enumerate(begun):
        table[b, :n] = ids[at:at + n]
        at += n
    return held, count, table, ids[at:], pages


def _check(h3, held, count, table, free, free_at, page, pages, tokens, most, bad=False):
    tab = _dev(table)
    want = O.kv_tables(held, count, table, free, free_at, page, pages, tokens, most)
    given = _dev([free_at])
    got = h3.kv_tables(_dev(held), _dev(count), tab, _dev(free), given, page, pages, tokens, most)
    assert got.cu_tokens.tolist() == want[0] and got.kv_len.tolist() == want[1]
    assert got.slots.tolist() == want[2] and got.positions.tolist() == want[3]
    assert np.array_equal(tab.cpu().numpy(), want[4]) and got.free_at.item() == want[5] and given.item() == free_at
    assert want[6] == bad and h3.h3fp4_device_error() == (512 if bad else 0)
    return got, tab


CASES = [   # held, new tokens, page
    ([0], [1], 16),
    ([0], [0], 64),
    ([15, 16, 17, 0], [1, 1, 1, 0], 16),
    ([0, 130, 7], [257, 0, 5_000], 128),
    ([31], [3_001], 32),
    ([100] * 64, [1] * 64, 64),
    (list(range(1_024)), [b % 3 for b in range(1_024)], 16),
    (list(range(1_025)), [1] * 1_025, 32),
    ([b % 77 for b in range(5_003)], [b % 5 for b in range(5_003)], 16),
]


@pytest.mark.parametrize("held,count,page", CASES)
@pytest.mark.parametrize("extra,free_at", [(0, 0), (5, 2)])
def test_against_one_token_after_another(h3, held, count, page, extra, free_at):
    rng = np.random.default_rng(len(held))
    h, c, table, free, pages = _inputs(rng, held, count, page, first=free_at)
    _check(h3, h, c, table, free, free_at, page, pages, int(c.sum()) + extra, int(c.max()))


def test_the_largest_batch(h3):
    rng = np.random.default_rng(5)
    held, count = rng.integers(0, 40, 65_535), rng.integers(0, 3, 65_535)
    h, c, table, free, pages = _inputs(rng, held, count, 16)
    _check(h3, h, c, table, free, 0, 16, pages, int(c.sum()) + 1_000, 2)


def test_long_sequences(h3):
    rng = np.random.default_rng(6)
    h, c, table, free, pages = _inputs(rng, [3_000_001, 0], [7, 300_000], 64)
    _check(h3, h, c, table, free, 0, 64, pages, 300_007, 300_000)


def test_no_sequences(h3):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    t = h3.kv_tables(none, none, none.view(0, 4), none, _dev([5]), 16, 9, 10, 0)
    assert t.cu_tokens.tolist() == [0] and t.free_at.item() == 5 and t.slots.tolist() == [-1] * 10
    assert t.positions.tolist() == [-1.0] * 10 and h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("copies", [1, 400])
def test_what_is_out_of_range_is_reported_and_left_out(h3, copies):
    """Alone, and in the middle of a batch of several tiles."""
    rng = np.random.default_rng(7)
    held, count = [5, 20, 0, 40] * copies, [3, 20, 17, 0] * copies
    h, c, table, free, pages = _inputs(rng, held, count, 16)
    args = dict(held=h, count=c, table=table, free=free, free_at=0, page=16, pages=pages, tokens=int(c.sum()), most=20)

    def change(name, at, value):
        a = args[name].copy()
        a[at] = value
        return {**args, name: a}

    mid = len(held) // 2 + 1 if copies > 1 else 1
    for bad in (change("held", mid, -1), change("count", mid, -3), change("count", mid, 21), change("held", mid, 10 ** 6),
                change("held", mid, 2 ** 31 - 5), change("free", 1, pages), change("free", 0, -1),
                {**args, "free": free[:2]}, {**args, "free_at": -1}, {**args, "free_at": len(free) + 4},
                {**args, "tokens": int(c.sum()) - 1}, {**args, "pages": int(table[mid, 1]) if table[mid, 1] > 0 else 1}):
        _check(h3, **bad, bad=True)
    _check(h3, **args)


def test_more_tokens_than_an_offset_holds(h3):
    """2,200 sequences of a million tokens: offsets stop at 2^31 - 1, rows past the arrays are not written."""
    n, page = 2_200, 128
    per = -(-1_000_000 // page)
    held, count = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n,), 1_000_000, dtype=torch.int32, device="cuda")
    table = torch.full((n, per), -1, dtype=torch.int32, device="cuda")
    t = h3.kv_tables(held, count, table, torch.arange(n * per, dtype=torch.int32, device="cuda"), _dev([0]), page, n * per, 4_000,
                     1_000_000)
    want = (torch.arange(n + 1, dtype=torch.int64) * 1_000_000).clamp(max=2 ** 31 - 1)
    assert torch.equal(t.cu_tokens.cpu().long(), want) and t.free_at.item() == n * per
    assert torch.equal(t.slots.cpu(), torch.arange(4_000)) and h3.h3fp4_device_error() == 512
    assert torch.equal(table.view(-1).cpu(), torch.arange(n * per, dtype=torch.int32))


def test_streams_outputs_given_and_graphs(h3):
    """A captured call follows lengths, pages and the free list's position on the device."""
    rng = np.random.default_rng(8)
    held, count = [30, 0, 64], [2, 50, 1]
    h, c, table, free, pages = _inputs(rng, held, count, 16, spare=40, room=8)
    dev = [_dev(a) for a in (h, c, table, free)]
    at, out_at = _dev([0]), _dev([0])
    buffers = dict(cu_tokens=_dev([0] * 4), kv_len=_dev([0] * 3), slots=torch.zeros(80, dtype=torch.int64, device="cuda"),
                   positions=torch.zeros(80, device="cuda"), free_at_out=out_at)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = h3.kv_tables(*dev, at, 16, pages, 80, 60, **buffers)
    assert got.slots is buffers["slots"]
    for lens, new, pos in (([30, 0, 64], [2, 50, 1], 0), ([32, 16, 5], [1, 0, 60], 3), ([0, 0, 0], [0, 0, 0], 1)):
        dev[0].copy_(_dev(lens))
        dev[1].copy_(_dev(new))
        dev[2].copy_(_dev(table))
        at.copy_(_dev([pos]))
        filled = np.where(table < 0, 0, table)
        dev[2].copy_(_dev(filled))
        want = O.kv_tables(lens, new, filled, free, pos, 16, pages, 80, 60)
        graph.replay()
        torch.cuda.synchronize()
        assert got.cu_tokens.tolist() == want[0] and got.kv_len.tolist() == want[1] and got.slots.tolist() == want[2]
        assert got.positions.tolist() == want[3] and np.array_equal(dev[2].cpu().numpy(), want[4]) and out_at.item() == want[5]
    assert h3.h3fp4_device_error() == 0


@pytest.mark.parametrize("free_at,wanted", [(-2, 10), (-2, 6), (-2, 2), (-2 ** 31, 10), (3, 10), (5, 1), (7, 2), (2 ** 31 - 1, 2)])
def test_no_page_is_taken_twice_whatever_the_place_in_the_list(h3, free_at, wanted):
    """A list of five pages taken from twice in a row, from before its beginning, past its end, and to its end."""
    free, page, at = np.array([5, 6, 7, 8, 9]), 16, free_at
    given = []
    for _ in range(2):
        table = np.full((1, wanted), -9)
        want = O.kv_tables([0], [wanted * page], table, free, at, page, 20, wanted * page, wanted * page)
        tab = _dev(table)
        got = h3.kv_tables(_dev([0]), _dev([wanted * page]), tab, _dev(free), _dev([at]), page, 20, wanted * page, wanted * page)
        assert np.array_equal(tab.cpu().numpy(), want[4]) and got.slots.tolist() == want[2]
        at = got.free_at.item()
        assert at == want[5] and free_at <= at <= max(5, free_at)
        assert h3.h3fp4_device_error() == (512 if want[6] else 0)
        given += [int(p) for p in tab.cpu().numpy()[0] if p >= 0]
    assert len(set(given)) == len(given)


@pytest.mark.parametrize("given", [False, True])
def test_tokens_without_any_row_are_reported(h3, given):
    kw = dict(slots=torch.empty(0, dtype=torch.int64, device="cuda"), positions=torch.empty(0, device="cuda")) if given else {}
    for count, bad in ((3, True), (0, False)):
        table = _dev([[-1]])
        t = h3.kv_tables(_dev([0]), _dev([count]), table, _dev([4, 5]), _dev([0]), 16, 9, 0, 3, **kw)
        assert t.cu_tokens.tolist() == [0, count] and t.free_at.item() == (1 if bad else 0) and t.slots.numel() == t.positions.numel() == 0
        assert table.item() == (4 if bad else -1) and h3.h3fp4_device_error() == (512 if bad else 0)
