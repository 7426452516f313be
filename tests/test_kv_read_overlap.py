"""Read-back into keys and values that share elements is refused, into ones
that are interleaved it is not."""
import ctypes

import numpy as np
import pytest
import torch

import dit_modulate_absmax_gb300 as pkg
from dit_modulate_absmax_gb300 import build as B

F = 0x100000              # a fake, 16-byte aligned "device" address (every call with one is refused)


@pytest.mark.parametrize("name,k,v", [
    ("the same", (0, 512, 128), (0, 512, 128)),
    ("one token on", (0, 512, 128), (512, 512, 128)),
    ("one head on", (0, 512, 128), (128, 512, 128)),
    ("within a row", (0, 512, 128), (64, 512, 128)),
    ("within an interleaved row", (0, 1024, 128), (384, 1024, 128)),
    ("within the gap and the next token", (0, 1024, 128), (640, 1024, 128)),
    ("before it", (512, 512, 128), (0, 512, 128)),
    ("other strides, ranges that overlap", (0, 1024, 128), (512, 512, 128)),
    ("heads outermost", (0, 128, 2560), (1280 - 64, 128, 2560)),
])
def test_shared_elements_are_refused(name, k, v):
    B.build()
    cache = pkg._KV_CACHE.pack(F, F, F, F, 4, 64, 4, 128)
    batch = pkg._KV_BATCH.pack(F, 4, F, F, 2, 5)
    at = [(ctypes.c_void_p(F + 2 * x[0]), *x[1:]) for x in (k, v)]
    assert pkg.lib().h3fp4_kv_cache_read(cache, batch, *at[0], *at[1], 10, None) == 4, name


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["token by token", "head by head", "heads outermost", "one token", "apart in one buffer"])
def test_interleaved_outputs_are_not(h3, layout):
    from test_gpu_kv_cache import _cache, _dev, _tables
    rng = np.random.default_rng(3)
    n, heads, dim = 1 if layout == "one token" else 37, 3, 64
    table, pages = _tables(rng, [n], 16)
    c = _cache(h3, rng, pages, heads, 16, dim)
    call = lambda **kw: h3.kv_cache_read(c, _dev(table), None, _dev([0, n]), n, n, **kw)
    shape, order = {"token by token": ((n, 2, heads, dim), lambda x: (x[:, 0], x[:, 1])),
                    "head by head": ((n, heads, 2, dim), lambda x: (x[:, :, 0], x[:, :, 1])),
                    "heads outermost": ((heads, 2, n, dim), lambda x: (x[:, 0].transpose(0, 1), x[:, 1].transpose(0, 1))),
                    "one token": ((n, heads, 2, dim), lambda x: (x[:, :, 0], x[:, :, 1])),
                    "apart in one buffer": ((2, n, heads, dim), lambda x: (x[0], x[1]))}[layout]
    wide = torch.full(shape, 7, dtype=torch.int16, device="cuda")
    k, v = order(wide)
    want = call()
    call(k=k, v=v)
    for got, ref in ((k, want[0]), (v, want[1])):
        assert torch.equal(got, ref.view(torch.int16))
    with pytest.raises(h3.H3FP4Error, match="UNSUPPORTED"):
        call(k=k, v=k)
    assert h3.h3fp4_device_error() == 0
