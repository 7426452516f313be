"""Bounded waits of the few-query attention, without a fault: copies that are
announced larger than they are never complete; the kernel must end soon after
its limit however many keys it had to read, with an error code, its outputs
untouched, and leave the device usable."""
import time

import numpy as np
import pytest
import torch

from test_gpu_kv_attention import _filled
from test_gpu_kv_cache import _dev

pytestmark = pytest.mark.gpu

LIMIT_US = 10_000


@pytest.mark.parametrize("lengths", [[777], [1_000_000], [40_000, 5, 20_000]])
def test_waits_run_out_once_then_device_recovers(h3, lengths):
    rng = np.random.default_rng(31)
    batch, heads, dim, page = len(lengths), 8, 128, 64
    pages = 100                                             # which the tables name many times
    table = rng.integers(0, pages, (batch, -(-max(lengths) // page))).astype(np.int32)
    c = _filled(h3, rng, np.arange(pages, dtype=np.int32)[None], [pages * page], pages, heads, page, dim)
    cu = np.arange(batch + 1)
    q = torch.randn(batch, heads, dim, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full((batch, heads), 7.0, device="cuda")
    most = max(lengths)
    arrays = _dev(table), _dev(lengths), _dev(cu)
    want = h3.kv_attention(q, c, *arrays, 1, most, return_lse=True)
    desc = h3._kv_batch(*arrays, 1, q.get_device())
    need = h3.h3fp4_kv_attention_workspace(batch, heads, heads, dim, batch, 1, most)
    ws = torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
    assert h3.h3fp4_device_error() == 0
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    h3.h3fp4_diag_attention_wait_timeout(q.data_ptr(), heads * dim, dim, out.data_ptr(), heads * dim, dim, lse.data_ptr(), batch,
                                         heads, c.struct(), desc, most, ws.data_ptr(), ws.numel(), LIMIT_US,
                                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    # three waits of a warp in turn, 10 ms each; twice that for what surrounds them (a wait for each unit of 32 keys would
    # take over a second with a million)
    assert elapsed < 0.06, f"the kernel returned only after {elapsed:.3f} s"
    assert h3.h3fp4_device_error() == 1024
    assert (out == 7).all() and (lse == 7).all(), "no output may be written when a wait gave up"
    got = h3.kv_attention(q, c, *arrays, 1, most, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert h3.h3fp4_device_error() == 0
