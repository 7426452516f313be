"""Attention over the 8-bit paged cache at the edges of what its arguments may
hold.  Bounds as in test_gpu_kv_attention where a test gives none of its own."""
import numpy as np
import pytest
import torch

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
