"""Attention over the 8-bit paged cache at the edges of what its arguments may
hold.  Bounds as in test_gpu_kv_attention where a test gives none of its own."""
import pytest
import torch

from test_gpu_kv_cache import _dev

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
