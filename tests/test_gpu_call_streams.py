"""Calls on a stream of the caller's: what a call allocates belongs to that
stream in torch's allocator, and calls on several streams keep apart."""
import numpy as np
import pytest
import torch

from test_gpu_kv_cache import _dev, _tables

pytestmark = pytest.mark.gpu


def _owner(address):
    """The stream whose pool holds this address."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in torch's pools")


def _bf16(*shape, seed=1):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def _attention_inputs(h3, new=140, length=2_000, heads=8, page=64, dim=128):
    table, pages = _tables(np.random.default_rng(3), [length], page)
    c = h3.KVCache.empty(pages, page, heads, dim)
    x = _bf16(length, heads, dim, seed=2)
    h3.kv_cache_write(c, x, x, _dev(table), _dev([0]), _dev([0, length]), length)
    return c, _dev(table), _dev([length]), _dev([0, new]), new, length


def test_attention_and_cache_allocate_on_the_calls_stream(h3, monkeypatch):
    c, table, length, cu, new, most = _attention_inputs(h3)
    q = _bf16(new, 8, 128)
    r = h3.Rope(torch.zeros(new, 1, device="cuda"), h3.rope_frequencies((128,)), (128,))
    seen = []
    call = h3.h3fp4_kv_attention
    monkeypatch.setattr(h3, "h3fp4_kv_attention", lambda *a: (seen.append(a[-3]), call(*a)))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse = h3.kv_attention(q, c, table, length, cu, new, most, return_lse=True, stream=s)
    k, v = h3.kv_cache_read(c, table, None, cu, new, new, stream=s)
    turned = h3.rope_axes(q, r, stream=s)
    assert seen[0] != 0                                    # a size whose workspace the call made itself
    assert {_owner(a) for a in (seen[0], *[t.data_ptr() for t in (out, lse, k, v, turned)])} == {s.cuda_stream}
    s.synchronize()
    plain = h3.kv_attention(q, c, table, length, cu, new, most, return_lse=True)
    assert _owner(seen[1]) == _owner(plain[0].data_ptr()) == torch.cuda.current_stream().cuda_stream
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])


def test_producers_and_gemm_allocate_on_the_calls_stream(h3):
    m, d = 256, 256
    x, gate, up = [_bf16(m, d, seed=i).view(torch.int16) for i in range(3)]
    mod = [(_bf16(1, d, seed=5 + i) * 0.1).view(torch.int16) for i in range(2)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [*h3.modulate_produce(x, *mod, [0, m], m, stream=s), *h3.swiglu_pack(gate, up, m, stream=s),
           *h3.quantize_pack(x, m, stream=s)]
    got.append(h3.modulate_absmax(x, *mod, [0, m], stream=s))
    got += h3.modulate_pack(x, *mod, [0, m], got[-1], m, stream=s)
    ts, packed, sfa = got[6:9]
    got.append(h3.gemm(packed, sfa, ts, packed, sfa, ts, m, stream=s))
    got.append(h3.swizzle_scales(torch.zeros(m, d // 16, dtype=torch.uint8, device="cuda"), stream=s))
    assert {_owner(t.data_ptr()) for t in got} == {s.cuda_stream}
    s.synchronize()
    want = h3.modulate_produce(x, *mod, [0, m], m)
    assert all(torch.equal(a, b) for a, b in zip(got[:2], want[:2]))


@pytest.mark.parametrize("new,length", [(140, 2_000), (1, 20_000)])
def test_calls_on_several_streams_and_allocations_meanwhile(h3, new, length):
    """Attention on two streams in turn, each with a workspace of the call's own, while the current stream allocates
    and fills blocks of the sizes that were just given back: the same bits as one call at a time."""
    args = _attention_inputs(h3, new, length)
    qs = [_bf16(new, 8, 128, seed=i) for i in range(2)]
    want = [h3.kv_attention(q, *args, causal=True)[0] for q in qs]
    need = h3.h3fp4_kv_attention_workspace(new, 8, 8, 128, 1, new, length)
    assert need > 0
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got, fill = [[], []], []
    for _ in range(20):
        for q, s, g in zip(qs, streams, got):
            g.append(h3.kv_attention(q, *args, causal=True, stream=s)[0])
            fill.append(torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda").sum())
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for g, w in zip(got, want) for o in g)
    assert all(int(f) == 0x7F * need for f in fill)
    assert h3.h3fp4_device_error() == 0
