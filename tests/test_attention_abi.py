"""Argument checks of the rotary, cache and attention entry points (CPU: every
call here is refused before anything is enqueued, or has nothing to do)."""
import numpy as np
import pytest

import dit_modulate_absmax_gb300 as pkg
from dit_modulate_absmax_gb300 import build as B
from oracle import attention as O

OK, NULL, ALIGN, SHAPE, UNSUP = 0, 1, 2, 3, 4
F, G = 0x10000, 0x90000000        # fake, 16-byte aligned "device" addresses (never dereferenced)


@pytest.fixture(scope="module")
def L():
    B.build()
    return pkg.lib()


def _rope(**kw):
    a = {**dict(positions=F, ld_positions=3, freqs=F, axes=3, dims=(44, 42, 42), layout=0, inverse=0), **kw}
    return pkg._ROPE.pack(a["positions"] or 0, a["ld_positions"], a["freqs"] or 0, a["axes"],
                          *(tuple(a["dims"]) + (0,) * 4)[:4], a["layout"], a["inverse"])


def _cache(**kw):
    a = {**dict(kc=F, vc=F, ks=F, vs=F, pages=4, page=64, heads=4, dim=128), **kw}
    return pkg._KV_CACHE.pack(a["kc"] or 0, a["vc"] or 0, a["ks"] or 0, a["vs"] or 0, a["pages"], a["page"], a["heads"],
                              a["dim"])


def _batch(**kw):
    a = {**dict(table=F, ld=4, len=F, cu=F, batch=2, most=5), **kw}
    return pkg._KV_BATCH.pack(a["table"] or 0, a["ld"], a["len"] or 0, a["cu"] or 0, a["batch"], a["most"])


def test_rope_refusals(L):
    def call(x=F, xt=512, xh=128, out=G, ot=512, oh=128, tokens=10, heads=4, dim=128, rope=None, **kw):
        r = _rope(**kw) if rope is None else rope
        return L.h3fp4_rope_axes(x, xt, xh, out, ot, oh, tokens, heads, dim, r, None)

    assert L.h3fp4_rope_axes(F, 512, 128, G, 512, 128, 10, 4, 128, None, None) == NULL
    assert call(x=None) == NULL and call(out=None) == NULL
    assert call(positions=None) == NULL and call(freqs=None) == NULL
    assert call(x=None, out=None, tokens=0) == OK and call(x=None, out=None, heads=0) == OK
    assert call(tokens=-1) == SHAPE and call(heads=-1) == SHAPE and call(heads=65536) == SHAPE
    assert call(dim=0) == SHAPE and call(dim=12) == SHAPE and call(dim=264) == SHAPE
    assert call(xt=-8) == SHAPE and call(xt=4) == ALIGN and call(x=F + 2) == ALIGN and call(oh=132) == ALIGN
    assert call(axes=0) == SHAPE and call(axes=5) == SHAPE
    assert call(dims=(43, 42, 42, 0)) == SHAPE and call(dims=(44, 44, 42, 0)) == SHAPE and call(dims=(-2, 42, 42, 0)) == SHAPE
    assert call(dims=(2**31 - 2, 2**31 - 2, 42, 0)) == SHAPE
    assert call(layout=2) == UNSUP and call(inverse=2) == SHAPE and call(ld_positions=2) == SHAPE
    assert call(positions=F + 2) == ALIGN and call(freqs=F + 4) == ALIGN
    assert call(ot=256) == SHAPE and call(oh=64) == SHAPE and call(ot=0) == SHAPE      # output rows that fold together
    assert call(out=F + 16) == UNSUP and call(out=F, ot=1024) == UNSUP                # overlapping, not in place


def test_cache_refusals(L):
    def write(c=None, b=None, k=F, kt=512, kh=128, v=F, vt=512, vh=128, tokens=10, rope=None):
        c, b = _cache() if c is None else c, _batch() if b is None else b
        return L.h3fp4_kv_cache_write(c, b, k, kt, kh, v, vt, vh, tokens,
                                      rope, None)

    def read(c=None, b=None, k=F, kt=512, kh=128, v=G, vt=512, vh=128, tokens=10):
        c, b = _cache() if c is None else c, _batch() if b is None else b
        return L.h3fp4_kv_cache_read(c, b, k, kt, kh, v, vt, vh, tokens, None)

    for f in (write, read):
        assert f(c=_cache(kc=None)) == NULL and f(c=_cache(vs=None)) == NULL
        assert f(c=_cache(page=48)) == UNSUP and f(c=_cache(page=256)) == UNSUP and f(c=_cache(dim=96)) == UNSUP
        assert f(c=_cache(heads=0)) == SHAPE and f(c=_cache(pages=-1)) == SHAPE
        assert f(c=_cache(kc=F + 8)) == ALIGN and f(c=_cache(ks=F + 2)) == ALIGN
        assert f(b=_batch(cu=None)) == NULL and f(b=_batch(table=None)) == NULL
        assert f(b=_batch(batch=-1)) == SHAPE and f(b=_batch(batch=65536)) == SHAPE and f(b=_batch(most=-1)) == SHAPE
        assert f(b=_batch(most=1_000_001)) == SHAPE and f(tokens=-1) == SHAPE and f(b=_batch(cu=F + 2)) == ALIGN
        assert f(kt=-8) == SHAPE and f(kt=12) == ALIGN and f(v=F + 4) == ALIGN
        assert f(tokens=0, k=None, v=None) == OK and f(b=_batch(batch=0)) == OK and f(b=_batch(most=0)) == OK
    assert write(k=None) == NULL and write(v=None) == NULL and write(b=_batch(len=None)) == NULL
    assert write(rope=_rope(dims=(128, 2, 0))) == SHAPE and write(rope=_rope(positions=None)) == NULL
    assert read(k=None, v=None) == NULL and read(kh=64) == SHAPE and read(vt=0) == SHAPE


def test_attention_refusals(L):
    def call(q=F, qt=1024, qh=128, out=G, ot=1024, oh=128, lse=None, tokens=10, heads=8, c=None, b=None, max_kv=256,
             scale=0.1, causal=1, window=0, ws=F, bytes=1 << 40):
        c, b = _cache() if c is None else c, _batch() if b is None else b
        return L.h3fp4_kv_attention(q, qt, qh, out, ot, oh, lse, tokens, heads, c, b, max_kv,
                                    scale, causal, window, ws, bytes, None)

    assert call(q=None) == NULL and call(out=None) == NULL and call(b=_batch(len=None)) == NULL
    assert call(heads=6) == SHAPE and call(heads=0) == SHAPE and call(max_kv=-1) == SHAPE and call(max_kv=2**30 + 1) == SHAPE
    assert call(window=-1) == SHAPE and call(causal=2) == SHAPE
    assert call(scale=float("nan")) == SHAPE and call(scale=float("inf")) == SHAPE
    assert call(c=_cache(page=8)) == UNSUP and call(out=F) == UNSUP and call(out=F + 128) == UNSUP
    assert call(q=F + 2) == ALIGN and call(lse=F + 2) == ALIGN and call(ws=F + 4) == ALIGN
    assert call(tokens=0, q=None, out=None) == OK and call(b=_batch(batch=0)) == OK
    w = L.h3fp4_kv_attention_workspace
    assert w(10, 6, 4, 128, 2, 5, 256) == -1 and w(10, 8, 4, 96, 2, 5, 256) == -1 and w(-1, 8, 4, 128, 2, 5, 256) == -1
    assert w(10, 8, 4, 128, 2, 5, 256) >= 0
    long = w(1, 8, 8, 128, 1, 1, 1 << 20)
    if long > 0:
        one = dict(b=_batch(batch=1, most=1), c=_cache(heads=8), tokens=1, max_kv=1 << 20)
        assert call(**one, ws=None) == NULL and call(**one, bytes=long - 1) == SHAPE


def test_workspace_grows_with_nothing_it_should_not(L):
    """No overflow at the largest sizes that are accepted."""
    for args in ((2**31 - 1, 65535, 1, 128, 65535, 1_000_000, 1 << 30), (1, 65535, 65535, 128, 1, 1, 1 << 30),
                 (2**31 - 1, 8, 8, 64, 65535, 1, 1 << 30)):
        assert -1 <= L.h3fp4_kv_attention_workspace(*args) < 1 << 60


def test_packed_structures_have_the_c_layout(tmp_path):
    """Sizes and member offsets of the header's structures, printed by a C program, against the packers'."""
    import os
    import struct
    import subprocess
    src = tmp_path / "layout.c"
    members = {"h3fp4_rope": ["positions", "ld_positions", "freqs", "axes", "dims", "layout", "inverse"],
               "h3fp4_kv_cache": ["k_codes", "v_codes", "k_scale", "v_scale", "num_pages", "page_size", "heads", "head_dim"],
               "h3fp4_kv_batch": ["page_table", "ld_table", "len", "cu_tokens", "batch", "max_tokens"]}
    lines = [f'printf("%zu\\n", sizeof({s}));' + "".join(f'printf("%zu\\n", offsetof({s}, {m}));' for m in ms)
             for s, ms in members.items()]
    src.write_text('#include <stdio.h>\n#include "h3fp4.h"\nint main(void) {' + "".join(lines) + "return 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout.split()]
    want = []
    for packer, kinds in ((pkg._ROPE, ["P", "q", "P", "i", "4i", "i", "i"]), (pkg._KV_CACHE, list("PPPPiiii")),
                          (pkg._KV_BATCH, list("PqPPii"))):
        want.append(packer.size)
        at = ""
        for k in kinds:
            want.append(struct.calcsize("@" + at + "0" + k[-1]))
            at += k
    assert got == want


def test_python_checks_before_any_pointer_is_taken():
    import torch
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                       # not on a device
        pkg.Rope(torch.zeros(2, 3), torch.zeros(64, dtype=torch.float64), (44, 42, 42))
    with pytest.raises(ValueError):
        pkg._need_tokens(x, "x")


def test_oracle_e4m3_pins():
    """Every code decodes and encodes to itself; midpoints go to the even code; saturation and NaN."""
    t = O.e4m3_table()
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    assert np.array_equal(O.e4m3_encode(t[codes]), codes)
    assert t[0x7E] == 448 and t[1] == 2.0 ** -9 and t[0x08] == 2.0 ** -6 and t[0x38] == 1.0
    for c in range(126):
        mid = (t[c] + t[c + 1]) / 2
        assert O.e4m3_encode(mid) == (c if c % 2 == 0 else c + 1)
        assert O.e4m3_encode(np.nextafter(mid, 1e9)) == c + 1 and O.e4m3_encode(np.nextafter(mid, 0)) == c
    assert O.e4m3_encode(1e9) == 0x7E and O.e4m3_encode(-1e9) == 0xFE and O.e4m3_encode(np.nan) == 0x7F
    assert O.e4m3_encode(np.inf) == 0x7F and O.e4m3_encode(-0.0) == 0x80


def test_oracle_scale_and_rotation_pins():
    assert O.block_scale(0.0) == 2.0 ** -40 and O.block_scale(448.0) == 1.0 and O.block_scale(449.0) == 2.0
    assert O.block_scale(3.4e38) == 2.0 ** 119 and O.block_scale(224.0) == 0.5
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1, 0, 0, 1]
    y, _ = O.rope(x, np.array([[1.0]]), np.array([np.pi / 2, np.pi]), (4,), "interleaved")
    assert np.allclose(y[0, 0], [0, 1, 0, -1])
    y, _ = O.rope(x, np.array([[1.0]]), np.array([np.pi / 2, np.pi]), (4,), "halves")
    assert np.allclose(y[0, 0], [0, 0, 1, -1])
    q, k = np.ones((2, 1, 2)), np.zeros((3, 1, 2))
    v = np.arange(6.0).reshape(3, 1, 2)
    out, lse, *_ = O.attention(q, k, v, 1.0, causal=True)
    assert np.allclose(out[:, 0], [[1, 2], [2, 3]]) and np.allclose(np.exp(lse[:, 0]), [2, 3])
