"""Argument checks of the norms with rotation, attention with sinks and with
shared prefixes, and the batch's tables (CPU: every call here is refused before
anything is enqueued, or has nothing to do)."""
import numpy as np
import pytest
import torch

import dit_modulate_absmax_gb300 as pkg
from dit_modulate_absmax_gb300 import build as B
from oracle import attention as O
from test_attention_abi import F, G, _batch, _cache, _rope

OK, NULL, ALIGN, SHAPE, UNSUP = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    B.build()
    return pkg.lib()


def _heads(**kw):
    a = {**dict(x=F, xt=512, xh=128, out=G, ot=512, oh=128, w=F, heads=4, wide=0), **kw}
    return pkg._NORM_HEADS.pack(a["x"] or 0, a["xt"], a["xh"], a["out"] or 0, a["ot"], a["oh"], a["w"] or 0, a["heads"], a["wide"])


def _grads(**kw):
    a = {**dict(dy=F, gt=512, gh=128, x=2 * F, xt=512, xh=128, dx=G, ot=512, oh=128, w=F, dw=F, heads=4, wide=0), **kw}
    return pkg._NORM_GRADS.pack(a["dy"] or 0, a["gt"], a["gh"], a["x"] or 0, a["xt"], a["xh"], a["dx"] or 0, a["ot"], a["oh"],
                                a["w"] or 0, a["dw"] or 0, a["heads"], a["wide"])


EPS = 1e-6


def test_norm_refusals(L):
    def call(q=None, k=None, tokens=10, dim=128, eps=EPS, rope=None, **kw):
        return L.h3fp4_norm_rope(_heads(**kw) if q is None else q, k, tokens, dim, eps, rope, None)

    assert call(x=None) == NULL and call(out=None) == NULL
    assert call(tokens=0, x=None, out=None) == OK and call(heads=0, x=None, out=None) == OK
    assert L.h3fp4_norm_rope(None, None, 10, 128, EPS, None, None) == OK
    assert call(tokens=-1) == SHAPE and call(dim=12) == SHAPE and call(dim=0) == SHAPE and call(dim=264) == SHAPE
    assert call(heads=-1) == SHAPE and call(heads=65536) == SHAPE and call(wide=2) == SHAPE
    for eps in (0.0, -1.0, 1e-31, 2e6, float("nan"), float("inf")):
        assert call(eps=eps) == SHAPE
    assert call(xt=-8) == SHAPE and call(xt=4) == ALIGN and call(x=F + 2) == ALIGN and call(oh=132) == ALIGN
    assert call(w=F + 1) == ALIGN and call(w=F + 2, wide=1) == ALIGN
    assert call(rope=_rope(inverse=1)) == SHAPE and call(rope=_rope(dims=(128, 2, 0))) == SHAPE
    assert call(rope=_rope(positions=None)) == NULL and call(rope=_rope(layout=2)) == UNSUP
    assert call(oh=64) == SHAPE and call(ot=256) == SHAPE                                   # output rows that fold together
    assert call(out=F + 16) == UNSUP and call(out=F, ot=1024) == UNSUP                      # overlapping, not in place
    k = _heads(x=F + 1024, out=G + 1024, xt=512)
    assert L.h3fp4_norm_rope(_heads(), k, 10, 128, EPS, None, None) == UNSUP                # k's output over q's
    assert call(k=_heads(x=None)) == NULL and call(k=_heads(heads=-1)) == SHAPE


def _overlap(a, ta, ha, na, b, tb, hb, nb, tokens, dim):
    at = [{p + t * st + h * sh + c for t in range(tokens) for h in range(n) for c in range(dim)}
          for p, st, sh, n in ((a, ta, ha, na), (b, tb, hb, nb))]
    return bool(at[0] & at[1])


@pytest.mark.parametrize("seed", range(6))
def test_overlap_of_queries_and_keys_is_found_where_rows_are_alike(L, seed):
    """Of two in-place sides with the same token stride: the call is refused exactly where they share an element.  (The call
    is given an output of the keys that is refused for another reason, so that nothing is ever enqueued: UNSUP comes first
    only where queries' output meets the keys' input.)"""
    rng = np.random.default_rng(seed)
    found = set()
    for _ in range(300):
        dim, tokens = 8 * int(rng.integers(1, 3)), int(rng.integers(1, 5))
        nq, nk = int(rng.integers(1, 5)), int(rng.integers(1, 5))
        head = dim + 8 * int(rng.integers(0, 3))
        if rng.integers(0, 2):
            token = head * (max(nq, nk) + int(rng.integers(0, 8)))
        else:                                                                              # heads outermost
            token = dim + 8 * int(rng.integers(0, 2))
            head = token * (tokens + int(rng.integers(0, 3)))
        shift = 8 * int(rng.integers(-20, 60))
        q = _grads(dy=F * 64, x=F * 64, dx=F * 64, gt=token, xt=token, ot=token, gh=head, xh=head, oh=head, heads=nq, dw=None)
        at = F * 64 + 2 * shift
        k = _grads(dy=G, x=at, dx=G, gt=token, xt=token, ot=token, gh=head, xh=head, oh=head, heads=nk, dw=F)
        want = _overlap(0, token, head, nq, shift, token, head, nk, tokens, dim)
        got = L.h3fp4_norm_rope_backward(q, k, tokens, dim, EPS, None, None, 0, None)     # no workspace: NULL if all else is well
        assert got == (UNSUP if want else NULL), (dim, tokens, nq, nk, head, token, shift)
        found.add(want)
    assert found == {True, False}


def test_norm_backward_refusals(L):
    def call(q=None, k=None, tokens=10, dim=128, eps=EPS, rope=None, ws=F, bytes=1 << 30, **kw):
        return L.h3fp4_norm_rope_backward(_grads(**kw) if q is None else q, k, tokens, dim, eps, rope, ws, bytes, None)

    need = L.h3fp4_norm_rope_backward_workspace(128)
    assert need > 0 and L.h3fp4_norm_rope_backward_workspace(12) == -1 and L.h3fp4_norm_rope_backward_workspace(512) == -1
    assert call(dy=None) == NULL and call(x=None) == NULL and call(dx=None) == NULL and call(ws=None) == NULL
    assert call(bytes=need - 1) == SHAPE and call(ws=F + 4) == ALIGN and call(dw=F + 2) == ALIGN
    assert call(tokens=0, dw=None, dy=None, x=None, dx=None) == OK and call(heads=0, dw=None) == OK
    assert call(eps=0.0) == SHAPE and call(rope=_rope(inverse=1)) == SHAPE and call(gt=4) == ALIGN and call(gh=-8) == SHAPE
    assert call(dx=F + 128) == UNSUP and call(dx=2 * F + 128) == UNSUP and call(oh=64) == SHAPE
    far = dict(dy=5 * F, x=6 * F, dx=G + (1 << 20))
    assert call(k=_grads(**far, dw=F + 64)) == UNSUP                                       # the weights' gradients overlap
    assert call(k=_grads(dy=5 * F, x=G, dx=G + (1 << 20), dw=None)) == UNSUP               # q's dx over k's x


def test_sinks_refusals(L):
    def call(q=F, out=G, tokens=10, heads=8, c=None, b=None, max_kv=256, window=9, sinks=4, ws=F, bytes=1 << 40):
        c, b = _cache() if c is None else c, _batch() if b is None else b
        return L.h3fp4_kv_attention_sinks(q, 1024, 128, out, 1024, 128, None, tokens, heads, c, b, max_kv, 0.1, 1, window, sinks, ws,
                                          bytes, None)

    assert call(sinks=-1) == SHAPE and call(sinks=2**30 + 1) == SHAPE and call(window=-1) == SHAPE
    assert call(q=None) == NULL and call(heads=6) == SHAPE and call(out=F) == UNSUP and call(c=_cache(page=8)) == UNSUP
    assert call(tokens=0) == OK and call(b=_batch(batch=0)) == OK and call(tokens=0, sinks=-1) == SHAPE


def test_shared_refusals(L):
    def call(q=F, out=G, tokens=10, heads=8, c=None, p=None, max_prefix=200, b=None, max_kv=256, scale=0.1, causal=1, ws=F,
             bytes=1 << 40):
        c, b, p = _cache() if c is None else c, _batch() if b is None else b, _batch() if p is None else p
        return L.h3fp4_kv_attention_shared(q, 1024, 128, out, 1024, 128, None, tokens, heads, c, p, max_prefix, b, max_kv, scale,
                                           causal, ws, bytes, None)

    assert L.h3fp4_kv_attention_shared(F, 1024, 128, G, 1024, 128, None, 10, 8, _cache(), None, 5, _batch(), 256, 0.1, 1, F, 1 << 40,
                                       None) == NULL
    for bad, status in ((dict(cu=None), NULL), (dict(len=None), NULL), (dict(table=None), NULL), (dict(batch=-1), SHAPE),
                        (dict(most=1_000_001), SHAPE), (dict(cu=F + 2), ALIGN)):
        assert call(p=_batch(**bad)) == status and call(b=_batch(**bad)) == status
    assert call(max_prefix=-1) == SHAPE and call(max_prefix=2**30 + 1) == SHAPE and call(max_kv=-1) == SHAPE
    assert call(q=None) == NULL and call(heads=6) == SHAPE and call(out=F) == UNSUP and call(causal=2) == SHAPE
    assert call(scale=float("nan")) == SHAPE and call(tokens=0) == OK and call(b=_batch(batch=0)) == OK and call(b=_batch(most=0)) == OK
    need = L.h3fp4_kv_attention_shared_workspace(10, 8, 4, 128, 2, 5, 200, 2, 5, 256)
    assert need >= 10 * 8 * 129 * 4 and call(ws=None) == NULL and call(bytes=need - 1) == SHAPE and call(ws=F + 8) == ALIGN
    w = L.h3fp4_kv_attention_shared_workspace
    assert w(10, 6, 4, 128, 2, 5, 200, 2, 5, 256) == -1 and w(10, 8, 4, 128, -1, 5, 200, 2, 5, 256) == -1
    assert w(10, 8, 4, 128, 2, 5, 200, 2, 5, -1) == -1 and w(0, 8, 4, 128, 2, 5, 200, 2, 5, 256) >= 0
    for args in ((2**31 - 1, 65535, 1, 128, 65535, 1_000_000, 1 << 30, 65535, 1_000_000, 1 << 30),
                 (2**31 - 1, 8, 8, 64, 1, 1_000_000, 1 << 30, 65535, 1, 1 << 30)):
        assert -1 <= w(*args) < 1 << 60


def _requests(**kw):
    a = {**dict(held=F, count=2 * F, table=3 * F, ld=4, free=4 * F, at=5 * F, at_out=6 * F, cu=7 * F, kv=8 * F, slots=9 * F,
                positions=10 * F, tokens=20, batch=3, most=10, num_free=9, pages=30, page=16), **kw}
    order = ("held", "count", "table", "ld", "free", "at", "at_out", "cu", "kv", "slots", "positions", "tokens", "batch", "most",
             "num_free", "pages", "page")
    return pkg._KV_REQUESTS.pack(*(a[n] or 0 for n in order))


def test_tables_refusals(L):
    def call(**kw):
        return L.h3fp4_kv_tables(_requests(**kw), None)

    assert L.h3fp4_kv_tables(None, None) == NULL
    for n in ("held", "count", "table", "free", "at", "at_out", "cu", "kv"):
        assert call(**{n: None}) == NULL, n
    for kw in (dict(batch=-1), dict(batch=65536), dict(most=-1), dict(most=1_000_001), dict(ld=-1), dict(tokens=-1), dict(tokens=2**31),
               dict(num_free=-1), dict(pages=-1)):
        assert call(**kw) == SHAPE, kw
    assert call(page=8) == UNSUP and call(page=48) == UNSUP
    assert call(held=F + 2) == ALIGN and call(slots=9 * F + 4) == ALIGN and call(cu=7 * F + 1) == ALIGN
    for kw in (dict(at_out=5 * F), dict(cu=F + 8), dict(kv=2 * F), dict(slots=4 * F + 32), dict(positions=9 * F + 152),
               dict(table=F), dict(table=7 * F - 44), dict(kv=7 * F + 12)):
        assert call(**kw) == UNSUP, kw


def test_packed_structures_have_the_c_layout(tmp_path):
    import os
    import struct
    import subprocess
    members = {"h3fp4_norm_heads": ["x", "x_token_stride", "x_head_stride", "out", "out_token_stride", "out_head_stride", "weight",
                                    "heads", "weight_f32"],
               "h3fp4_norm_grads": ["dy", "dy_token_stride", "dy_head_stride", "x", "x_token_stride", "x_head_stride", "dx",
                                    "dx_token_stride", "dx_head_stride", "weight", "dweight", "heads", "weight_f32"],
               "h3fp4_kv_requests": ["held", "count", "page_table", "ld_table", "free_pages", "free_at", "free_at_out", "cu_tokens",
                                     "kv_len", "slots", "positions", "tokens", "batch", "max_tokens", "num_free", "num_pages",
                                     "page_size"]}
    lines = [f'printf("%zu\\n", sizeof({s}));' + "".join(f'printf("%zu\\n", offsetof({s}, {m}));' for m in ms)
             for s, ms in members.items()]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "h3fp4.h"\nint main(void) {' + "".join(lines) + "return 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout.split()]
    want = []
    for packer, kinds in ((pkg._NORM_HEADS, "PqqPqqPii"), (pkg._NORM_GRADS, "PqqPqqPqqPPii"), (pkg._KV_REQUESTS, "PPPqPPPPPPPqiiiii")):
        want.append(packer.size)
        for i, k in enumerate(kinds):
            want.append(struct.calcsize("@" + kinds[:i] + "0" + k))
    assert got == want


def test_integers_past_32_bits_are_refused(L):
    big = 1 << 32
    with pytest.raises(pkg.H3FP4Error):
        pkg.h3fp4_kv_attention_sinks(F, 1024, 128, G, 1024, 128, None, 10, 8, _cache(), _batch(), 256, 0.1, 1, 9, big + 4, F, 1 << 40)
    with pytest.raises(pkg.H3FP4Error):
        pkg.h3fp4_kv_attention_shared(F, 1024, 128, G, 1024, 128, None, 10, 8, _cache(), _batch(), big + 5, _batch(), 256, 0.1, 1, F, 1)
    with pytest.raises(pkg.H3FP4Error):
        pkg.h3fp4_norm_rope(None, None, 0, big + 128, EPS)
    with pytest.raises(pkg.H3FP4Error):
        pkg.h3fp4_norm_rope_backward_workspace(big + 128)


class _On:
    """A tensor that says it lies on CUDA device `device` (checks come before any address is used)."""

    def __init__(self, t, device):
        self.t, self.at = t, device

    def get_device(self):
        return self.at

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_tensors_of_several_devices_and_wrong_kinds_are_refused():
    x = _On(torch.zeros(2, 4, 128, dtype=torch.bfloat16), 0)
    other = _On(torch.zeros(2, 4, 128, dtype=torch.bfloat16), 1)
    w = _On(torch.ones(128), 0)
    for kw in (dict(k=other), dict(q_weight=_On(torch.ones(128), 1)), dict(q_weight=_On(torch.ones(64), 0)),
               dict(q_weight=_On(torch.ones(128, dtype=torch.float64), 0)), dict(q_weight=_On(torch.ones(256)[::2], 0)),
               dict(q_out=other), dict(k_weight=w), dict(k=_On(torch.zeros(3, 4, 128, dtype=torch.bfloat16), 0)),
               dict(k=_On(torch.zeros(2, 4, 64, dtype=torch.bfloat16), 0))):
        with pytest.raises(ValueError):
            pkg.norm_rope(x, **kw)
    with pytest.raises(ValueError):
        pkg.norm_rope_backward(other, None, x, q_out=x)
    with pytest.raises(ValueError):
        pkg.norm_rope_backward(x, x, x, q_out=x)
    with pytest.raises(ValueError):
        pkg.norm_rope_backward(x, None, x, q_out=x, q_weight_grad=w)
    n, at = _On(torch.zeros(3, dtype=torch.int32), 0), _On(torch.zeros(1, dtype=torch.int32), 0)
    table, free = _On(torch.zeros(3, 4, dtype=torch.int32), 0), _On(torch.zeros(5, dtype=torch.int32), 0)
    for args in ((n, n, _On(table.t, 1), free, at), (n, _On(torch.zeros(2, dtype=torch.int32), 0), table, free, at),
                 (n, n, table, free, n), (n, n, table, _On(torch.zeros(5, dtype=torch.int64), 0), at)):
        with pytest.raises(ValueError):
            pkg.kv_tables(*args, 16, 9, 10, 5)
    for kw in (dict(tokens=1 << 31), dict(page_size=(1 << 32) + 16), dict(max_tokens=1 << 31)):
        with pytest.raises(pkg.H3FP4Error):
            pkg.kv_tables(n, n, table, free, at, **{**dict(page_size=16, num_pages=9, tokens=10, max_tokens=5), **kw})


def test_oracle_pins():
    """Closed forms of the oracle's own additions."""
    y, _ = O.norm_rope(np.array([[[3.0, 4.0]]]), np.array([1.0, 2.0]), 0.0, lambda z: (z, np.abs(z)))
    assert np.allclose(y[0, 0], np.array([3, 8]) / np.sqrt(12.5))
    dx, dw, _, _ = O.norm_rope_backward(np.array([[[1.0, 0.0]]]), np.array([[[3.0, 4.0]]]), np.ones(2), 0.0, lambda z: (z, np.abs(z)))
    r = 1 / np.sqrt(12.5)
    assert np.allclose(dw, [3 * r, 0]) and np.allclose(dx[0, 0], [r - 3 * r * 3 * r * r / 2, -4 * r * 3 * r * r / 2])
    q, k, v = np.zeros((1, 1, 2)), np.zeros((6, 1, 2)), np.eye(6)[:, None, :2] + np.arange(6.0)[:, None, None]
    out, lse, *_ = O.attention(q, k, v, 1.0, causal=True, window=2, sinks=1)        # keys 0, 4, 5
    assert np.allclose(np.exp(lse), 3) and np.allclose(out[0, 0], [10 / 3, 9 / 3])
    out, lse, *_ = O.attention(q, k, v, 1.0, causal=True, before=4)                 # a prefix of 4, then two keys of its own
    assert np.allclose(np.exp(lse), 6)
    out, lse, *_ = O.attention(np.zeros((3, 1, 2)), k, v, 1.0, causal=True, before=4)
    assert np.allclose(np.exp(lse[:, 0]), [4, 5, 6])                                # the first query stands before its own keys
    got = O.kv_tables([3, 0], [2, 5], np.array([[7, -1], [-1, -1]]), [9, 8, 6], 0, 4, 10, 8, 5)
    assert got[0] == [0, 2, 7] and got[1] == [5, 5] and got[2] == [31, 36, 32, 33, 34, 35, 24, -1]
    assert got[3] == [3, 4, 0, 1, 2, 3, 4, -1] and got[4].tolist() == [[7, 9], [8, 6]] and got[5] == 3 and not got[6]
