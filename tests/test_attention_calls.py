"""The Python calls of the cache and its attention (CPU): what they check and
pass on, with tensors that are stand-ins and entry points that only record."""
import struct

import pytest
import torch

import dit_modulate_absmax_gb300 as pkg
from dit_modulate_absmax_gb300 import build as B


class Fake:
    """A contiguous device tensor as far as the calls look at one."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.int32, device=0, at=0x10000, stride=None):
        self.shape, self.dtype, self._device, self._at = torch.Size(shape), dtype, device, at
        self.device = torch.device("cuda", device)
        self._stride = stride or torch.empty(shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def is_contiguous(self):
        return self._stride == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return self._at

    def get_device(self):
        return self._device

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


class FakeStream:
    cuda_stream = 0


def _cache(device=0, **other):
    d = {n: device for n in ("kc", "ks", "vc", "vs")} | other
    return pkg.KVCache(Fake(4, 2, 16, 64, dtype=torch.uint8, device=d["kc"]), Fake(4, 2, dtype=torch.float32, device=d["ks"]),
                       Fake(4, 2, 16, 64, dtype=torch.uint8, device=d["vc"]), Fake(4, 2, dtype=torch.float32, device=d["vs"]))


def _x(tokens=3, heads=2, device=0, at=0x10000):
    return Fake(tokens, heads, 64, dtype=torch.bfloat16, device=device, at=at)


@pytest.fixture(autouse=True)
def built():
    B.build()


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the C entry points that were reached; the current stream of a device is its number."""
    got = []
    for name in ("h3fp4_rope_axes", "h3fp4_kv_cache_write", "h3fp4_kv_cache_read", "h3fp4_kv_attention"):
        monkeypatch.setattr(pkg, name, lambda *a, name=name: got.append((name, a)))
    monkeypatch.setattr(pkg, "_raw_stream", lambda stream, t: t.get_device())
    return got


def test_workspace_of_one_device_is_not_anothers(calls, monkeypatch):
    """Devices may differ in their SMs, and with them the parts of the keys."""
    sizes = {0: 1_000, 1: 5_000}
    device = [0]
    monkeypatch.setattr(pkg, "h3fp4_kv_attention_workspace", lambda *a: sizes[device[0]])
    made = []
    monkeypatch.setattr(pkg, "_empty", lambda stream, n, dtype, device: (made.append(n), Fake(n, dtype=dtype))[1])
    pkg._attention_workspace.cache_clear()
    for device[0] in (0, 1, 0, 1):
        d = device[0]
        pkg.kv_attention(_x(device=d), _cache(d), Fake(1, 4, device=d), Fake(1, device=d), Fake(2, device=d), 3, 64,
                         out=_x(device=d, at=0x90000))
    pkg._attention_workspace.cache_clear()
    assert made == [1_000, 5_000, 1_000, 5_000]


@pytest.mark.parametrize("name,value", [("window", 2**32 + 5), ("window", -2**32), ("max_kv", 2**32 + 64), ("max_kv", 2**31),
                                        ("max_tokens", 2**32 + 3), ("causal", 2**32)])
def test_integers_that_do_not_fit_are_refused(name, value):
    """... and not cut to 32 bits (the call has no tokens, so that it would do nothing if it were let through)."""
    kw = {"max_tokens": 3, "max_kv": 64, "causal": 0, "window": 0} | {name: value}
    most, kv = kw.pop("max_tokens"), kw.pop("max_kv")
    with pytest.raises((pkg.H3FP4Error, ValueError, struct.error)):
        pkg.kv_attention(_x(0), _cache(), Fake(1, 4), Fake(1), Fake(2), most, kv, out=_x(0, at=0x90000), stream=FakeStream(), **kw)


@pytest.mark.parametrize("call", ["h3fp4_kv_attention_workspace", "h3fp4_rope_axes"])
def test_integers_of_the_mirrors_that_do_not_fit_are_refused(call):
    sizes = [1, 8, 8, 64, 1, 1, 100]
    with pytest.raises(pkg.H3FP4Error):
        if call == "h3fp4_rope_axes":
            rope = pkg._ROPE.pack(0x10000, 1, 0x10000, 1, 0, 0, 0, 0, 0, 0)
            pkg.h3fp4_rope_axes(0x10000, 128, 64, 0x90000, 128, 64, 0, 2**32 + 2, 64, rope)
        else:
            pkg.h3fp4_kv_attention_workspace(*sizes[:6], 2**32 + 100)


def test_tensors_of_one_call_lie_on_one_device(calls):
    ok = [Fake(1, 4), Fake(1), Fake(2)]
    pos, freqs = dict(dtype=torch.float32), dict(dtype=torch.float64)
    rope = lambda d=0: pkg.Rope(Fake(3, 1, device=d, **pos), Fake(32, device=d, **freqs), (64,))
    pkg.kv_attention(_x(), _cache(), *ok, 3, 64, out=_x(at=0x90000), workspace=Fake(1 << 20, dtype=torch.uint8))
    pkg.kv_cache_write(_cache(), _x(), _x(), *ok, 3, rope=rope())
    pkg.kv_cache_write(_cache(), _x(), _x(), *ok, 3)
    pkg.kv_cache_read(_cache(), *ok, 3, 3, k=_x(), v=_x(at=0x90000))
    pkg.kv_cache_read(_cache(), ok[0], None, ok[2], 3, 3, k=_x(), v=_x(at=0x90000))
    pkg.rope_axes(_x(), rope(), out=_x(at=0x90000))
    assert len(calls) == 6
    for name in ("kc", "ks", "vc", "vs"):
        with pytest.raises(ValueError):
            _cache(**{name: 1})
    with pytest.raises(ValueError):
        pkg.Rope(Fake(3, 1, device=1, **pos), Fake(32, **freqs), (64,))
    for i in range(3):
        arrays = list(ok)
        arrays[i] = Fake(*ok[i].shape, device=1)
        for call in (lambda: pkg.kv_attention(_x(), _cache(), *arrays, 3, 64, out=_x(at=0x90000)),
                     lambda: pkg.kv_cache_write(_cache(), _x(), _x(), *arrays, 3),
                     lambda: pkg.kv_cache_read(_cache(), *arrays, 3, 3, k=_x(), v=_x(at=0x90000))):
            with pytest.raises(ValueError):
                call()
    far, out = _x(device=1), _x(at=0x90000)
    lse = Fake(3, 2, dtype=torch.float32, device=1)
    for call in (lambda: pkg.kv_attention(_x(), _cache(1), *ok, 3, 64, out=out), lambda: pkg.kv_attention(_x(), _cache(), *ok, 3, 64, out=far),
                 lambda: pkg.kv_attention(_x(), _cache(), *ok, 3, 64, out=out, lse=lse),
                 lambda: pkg.kv_attention(_x(), _cache(), *ok, 3, 64, out=out, workspace=Fake(1 << 20, dtype=torch.uint8, device=1)),
                 lambda: pkg.kv_cache_write(_cache(1), _x(), _x(), *ok, 3), lambda: pkg.kv_cache_write(_cache(), _x(), far, *ok, 3),
                 lambda: pkg.kv_cache_write(_cache(), _x(), _x(), *ok, 3, rope=rope(1)),
                 lambda: pkg.kv_cache_read(_cache(1), *ok, 3, 3, k=_x(), v=out), lambda: pkg.kv_cache_read(_cache(), *ok, 3, 3, k=_x(), v=far),
                 lambda: pkg.rope_axes(_x(), rope(), out=far), lambda: pkg.rope_axes(_x(), rope(1), out=out)):
        with pytest.raises(ValueError):
            call()
    assert len(calls) == 6


@pytest.mark.parametrize("shape,stride", [((1 << 20,), (0,)), ((1 << 10, 1 << 10), (1 << 11, 1)), ((1 << 20,), (2,))])
def test_a_workspace_with_gaps_is_refused(calls, shape, stride):
    """Its bytes are counted by its elements and written one after another: an expanded one has fewer, one with gaps has
    someone else's between."""
    with pytest.raises(ValueError, match="workspace"):
        pkg.kv_attention(_x(), _cache(), Fake(1, 4), Fake(1), Fake(2), 3, 64, out=_x(at=0x90000),
                         workspace=Fake(*shape, dtype=torch.uint8, stride=stride))
    assert not calls


def test_a_cache_or_rotation_does_not_change_its_tensors():
    """The addresses that the kernels get are those of the tensors it was made of: another tensor put in their place would
    be ignored, and the old one's memory used after it is freed."""
    rope = pkg.Rope(Fake(3, 1, dtype=torch.float32), Fake(32, dtype=torch.float64), (64,))
    cache = _cache()
    for of, names in ((rope, ("positions", "freqs", "dims", "layout")), (cache, ("k_codes", "k_scale", "v_codes", "v_scale", "heads"))):
        for name in names:
            before = getattr(of, name)
            with pytest.raises(AttributeError):
                setattr(of, name, before)
            assert getattr(of, name) is before
    assert (cache.num_pages, cache.heads, cache.page_size, cache.head_dim) == (4, 2, 16, 64)
    assert (rope.dims, rope.layout) == ((64,), "interleaved")


def test_wait_diagnostic_refusals():
    """Arguments that are refused before anything is enqueued."""
    F, G = 0x100000, 0x90000000
    L = pkg.lib()

    def call(q=F, heads=8, dim=128, most=1, limit=1000, ws=F, have=1 << 40, max_kv=256):
        cache = pkg._KV_CACHE.pack(F, F, F, F, 4, 64, 8, dim)
        return L.h3fp4_diag_attention_wait_timeout(q, heads * dim, dim, G, heads * dim, dim, None, 2, heads, cache,
                                                   pkg._KV_BATCH.pack(F, 4, F, F, 2, most), max_kv, ws, have, limit, None)

    assert call(q=None) == 1 and call(heads=12) == 3 and call(limit=0) == 3 and call(limit=2_000_001) == 3
    assert call(heads=72) == 4 and call(most=9) == 4 and call(dim=64) == 4 and call(max_kv=-1) == 3
    assert call(max_kv=1 << 20, ws=None) == 1 and call(max_kv=1 << 20, have=16) == 3
