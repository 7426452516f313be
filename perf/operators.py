"""Work over the attention operators: rotary positions with several axes, the
8-bit key/value cache (written, read back) and the attention that reads it.

With ``own`` false every operator is computed in its plain form, elementary
torch operations in 32 bits rounded once at the end; with ``own`` true the
same pass makes the calls a user makes of this framework.  Sizes are those of
the streaming DiT block (37,810 tokens, of which 32,768 are cached and 5,042
are new; 56 heads of 128) and generic ones for token-by-token decoding.
"""
import math

import torch

own = False

E_MIN, E_MAX = -40, 119          # exponents a cache block's power-of-two scale may take
LAYOUTS = ("interleaved", "halves")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token's queries and keys, all heads (latency of a decoding step)
        dict(name="rope_token", op="rope", tokens=1, heads=112, dim=128, d0=44, d1=42, d2=42, layout=0, inverse=0, ld=168),
        # the whole video's queries and keys, read from the QKV projection's rows
        dict(name="rope_video", op="rope", tokens=37_810, heads=112, dim=128, d0=32, d1=48, d2=48, layout=0, inverse=0,
             ld=168),
        # gradient of a chunk's queries; pairs split in halves, sections that are no multiple of eight
        dict(name="rope_grad_halves", op="rope", tokens=5_042, heads=56, dim=128, d0=44, d1=42, d2=42, layout=1,
             inverse=1, ld=56),
        # a decoding step of 64 requests: one token each into blocks that already hold some
        dict(name="cache_append", op="write", batch=64, new=1, old=4_095, heads=8, dim=128, page=16, rope=0, read=0),
        # prompts of several lengths, written to empty and half-filled blocks
        dict(name="cache_prompts", op="write", batch=5, new=3_001, old=77, heads=16, dim=64, page=32, rope=0, read=0),
        # a video chunk after its 32,768 cached tokens: keys rotated as they are written, the blocks read back
        dict(name="cache_chunk", op="write", batch=1, new=5_042, old=32_768, heads=56, dim=128, page=64, rope=1, read=1),
        # the whole video's keys and values read back to bf16
        dict(name="cache_read_video", op="read", batch=1, tokens=37_810, heads=56, dim=128, page=64),
        # one short request decoding
        dict(name="attn_token", op="attn", batch=1, q=1, kv=777, heads=56, kv_heads=56, dim=128, page=16, causal=1,
             window=0, lse=0),
        # a batch of 32 ragged requests decoding, eight query heads to a key head
        dict(name="attn_decode_batch", op="attn", batch=32, q=1, kv=8_190, heads=64, kv_heads=8, dim=128, page=64,
             causal=1, window=0, lse=0),
        # one very long request decoding
        dict(name="attn_decode_long", op="attn", batch=1, q=1, kv=262_143, heads=32, kv_heads=8, dim=128, page=128,
             causal=1, window=0, lse=1),
        # ragged prompts, causal with a sliding window, four query heads to a key head
        dict(name="attn_prompts", op="attn", batch=6, q=2_050, kv=2_500, heads=16, kv_heads=4, dim=64, page=32, causal=1,
             window=1_000, lse=1),
        # the video chunk against everything cached, itself included
        dict(name="attn_chunk", op="attn", batch=1, q=5_042, kv=37_810, heads=56, kv_heads=56, dim=128, page=64,
             causal=0, window=0, lse=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn"])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        heads = rng.randint(1, 112)
        d1 = 2 * rng.randint(1, dim // 6)
        d0 = dim - 2 * d1 - rng.choice([0, 0, 8])
        return dict(op=op, tokens=_log(rng, 1, 37_810), heads=heads, dim=dim, d0=d0, d1=d1, d2=d1,
                    layout=rng.randint(0, 1), inverse=rng.randint(0, 1), ld=heads + rng.randint(0, 56))
    if op == "write":
        heads = rng.randint(1, 56)
        new = rng.choice([1, _log(rng, 1, 5_042)])
        return dict(op=op, batch=_log(rng, 1, 64) if new <= 64 else 1 + 20_000 // (new * 4), new=new,
                    old=_log(rng, 1, 4_095) - 1, heads=heads, dim=dim, page=page, rope=rng.randint(0, 1), read=1)
    if op == "read":
        tokens = _log(rng, 1, 37_810)
        return dict(op=op, batch=max(1, min(_log(rng, 1, 64), 37_810 // tokens)), tokens=tokens, heads=rng.randint(1, 56),
                    dim=dim, page=page)
    kv_heads = rng.randint(1, 8)
    group = rng.choice([1, 2, 4, 5, 8])
    q = rng.choice([1, 1, _log(rng, 2, 24), _log(rng, 2, 5_042)])
    batch = _log(rng, 1, 32) if q <= 24 else rng.randint(1, 4)
    kv = max(q, min(_log(rng, 16, 65_536), 4_000_000_000 // (batch * q * kv_heads * group), 2_000_000 // batch))
    return dict(op="attn", batch=batch, q=q, kv=kv, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page,
                causal=rng.randint(0, 1), window=rng.choice([0, 0, _log(rng, 1, 4_096)]), lse=rng.randint(0, 1))


def _ragged(most, batch):
    """Lengths of a batch: the first is the longest, the others spread down to a quarter of it."""
    return [max(1, round(most * (1 - 0.75 * ((b * 0.6180339887498949) % 1.0)))) if most else 0 for b in range(batch)]


def _attn_lengths(c):
    qs = _ragged(c["q"], c["batch"])
    return qs, [max(k, n) for k, n in zip(_ragged(c["kv"], c["batch"]), qs)]


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 4 * n + 12 * c["tokens"], "flops": 3 * n}
    if c["op"] == "write":
        new, old = _ragged(c["new"], c["batch"]), _ragged(c["old"], c["batch"])
        width = c["heads"] * c["dim"]
        blocks = sum((o + n - 1) // c["page"] - o // c["page"] + 1 for o, n in zip(old, new))
        held = sum(o % c["page"] for o in old)                    # tokens of half-filled blocks: read, perhaps re-encoded
        got = 2 * width * (2 * sum(new) + sum(new) + held) + 16 * blocks * c["heads"]
        back = 2 * width * 3 * (sum(new) + held) if c["read"] else 0
        return {"bytes": got + back + (12 * sum(new) if c["rope"] else 0), "flops": 4 * width * sum(new)}
    if c["op"] == "read":
        n = sum(_ragged(c["tokens"], c["batch"])) * c["heads"] * c["dim"]
        return {"bytes": 2 * 3 * n, "flops": 2 * n}
    qs, ks = _attn_lengths(c)
    pairs = keys = 0
    for n, L in zip(qs, ks):
        first = L - n                                              # position of the first query
        low = max(0, first - c["window"] + 1) if c["window"] else 0
        keys += L - low
        for lo, hi, sign in ((first + 1, L, 1), (first + 1 - c["window"], L - c["window"], -1)):
            if sign > 0:
                pairs += (lo + hi) * (hi - lo + 1) // 2 if c["causal"] else n * L
            elif c["window"] and hi > 0:
                lo = max(lo, 1)
                pairs -= (lo + hi) * (hi - lo + 1) // 2
    rows = sum(qs) * c["heads"] * c["dim"]
    return {"bytes": 4 * rows + 2 * keys * c["kv_heads"] * c["dim"] + (4 * sum(qs) * c["heads"] if c["lse"] else 0),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _positions(tokens, gen):
    """Time, height and width of a video's tokens, 45 x 80 patches a frame, from a frame of the seed."""
    first = int(torch.randint(0, 32, (1,), generator=gen, device="cuda"))
    i = torch.arange(tokens, device="cuda")
    return torch.stack([first + i // 3600, i // 80 % 45, i % 80], dim=1).float()


def _frequencies(dims):
    """Radians per unit of position for each rotated pair, 10000^(-2j/d) along each axis."""
    return torch.cat([10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in dims]).cuda()


def _tables(lengths, page, gen):
    """Page tables of a batch over pages in random order, and the number of pages."""
    counts = [-(-n // page) for n in lengths]
    ids = torch.randperm(sum(counts) + 3, generator=gen, device="cuda").int()
    table = torch.zeros(len(lengths), max(1, max(counts)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(counts) + 3


def _filled(pages, heads, page, dim, gen):
    """Codes and scales of a cache in use: values near N(0, 1), scales of several blocks apart by powers of two."""
    def one():
        codes = torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda")
        for i in range(0, pages, 256):
            n = min(256, pages - i)
            x = torch.randn(n, heads, page, dim, generator=gen, device="cuda") * 64
            codes[i:i + n] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = torch.exp2(torch.randint(-7, -4, (pages, heads), generator=gen, device="cuda").float())
        return codes, scale
    (kc, ks), (vc, vs) = one(), one()
    return kc, ks, vc, vs


def _cu(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).int()


def _bf16(shape, gen, scale=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for i in range(0, shape[0], 4096):
        n = min(4096, shape[0] - i)
        x[i:i + n] = (torch.randn(n, *shape[1:], generator=gen, device="cuda") * scale).bfloat16()
    return x


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        dims = (c["d0"], c["d1"], c["d2"])
        wide = _bf16((c["tokens"], c["ld"], c["dim"]), gen)
        s |= {"x": wide[:, :c["heads"]], "positions": _positions(c["tokens"], gen), "freqs": _frequencies(dims), "dims": dims}
        return s
    if c["op"] == "write":
        new, old = _ragged(c["new"], c["batch"]), _ragged(c["old"], c["batch"])
        total = sum(new)
        table, pages = _tables([n + o for n, o in zip(new, old)], c["page"], gen)
        wide = _bf16((total, 3 * c["heads"], c["dim"]), gen, 1.5)   # the rows of a QKV projection
        s |= {"k": wide[:, c["heads"]:2 * c["heads"]], "v": wide[:, 2 * c["heads"]:], "table": table,
              "cache": _filled(pages, c["heads"], c["page"], c["dim"], gen), "old": torch.tensor(old, device="cuda").int(),
              "cu": _cu(new), "new": max(new), "from": torch.tensor([o - o % c["page"] for o in old], device="cuda").int()}
        back = [n + o % c["page"] for n, o in zip(new, old)]
        s |= {"back": _cu(back), "back_total": sum(back), "back_most": max(back)}
        if c["rope"]:
            d1 = c["dim"] // 16 * 6
            dims = (c["dim"] - 2 * d1, d1, d1)
            s |= {"positions": _positions(total, gen), "freqs": _frequencies(dims), "dims": dims}
        return s
    if c["op"] == "read":
        n = _ragged(c["tokens"], c["batch"])
        table, pages = _tables(n, c["page"], gen)
        return s | {"table": table, "cache": _filled(pages, c["heads"], c["page"], c["dim"], gen), "back": _cu(n),
                    "back_total": sum(n), "back_most": max(n), "from": torch.zeros(len(n), dtype=torch.int32, device="cuda")}
    qs, ks = _attn_lengths(c)
    table, pages = _tables(ks, c["page"], gen)
    return s | {"q": _bf16((sum(qs), c["heads"], c["dim"]), gen, 2.0), "table": table, "cu": _cu(qs), "most": max(qs),
                "cache": _filled(pages, c["kv_heads"], c["page"], c["dim"], gen),
                "kv": torch.tensor(ks, device="cuda").int(), "kv_most": max(ks)}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _rotate(x, positions, freqs, dims, layout, inverse):
    """x [tokens, heads, dim] rotated pair by pair, in 32 bits."""
    halves = [d // 2 for d in dims]
    axis = torch.repeat_interleave(torch.arange(3, device=x.device), torch.tensor(halves, device=x.device))
    start = torch.tensor([0, dims[0], dims[0] + dims[1]], device=x.device)[axis]
    j = torch.arange(sum(halves), device=x.device) - start // 2
    half = torch.tensor(halves, device=x.device)[axis]
    lo = start + (2 * j if layout == 0 else j)
    hi = lo + (1 if layout == 0 else half)
    angle = positions[:, axis] * freqs.float() * (-1 if inverse else 1)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    y = x.float()
    a, b = y[:, :, lo], y[:, :, hi]
    y[:, :, lo] = a * cos - b * sin
    y[:, :, hi] = a * sin + b * cos
    return y.bfloat16()


def _plain_write(s, c, x, codes, scales):
    """One of keys and values into its codes and scales: the touched blocks as a whole."""
    page = c["page"]
    n = s["cu"][1:] - s["cu"][:-1]
    first = s["old"] // page
    blk = first[:, None] + torch.arange(s["new"] // page + 2, device="cuda")
    seq, at = torch.nonzero((blk * page < (s["old"] + n)[:, None]) & (n > 0)[:, None], as_tuple=True)
    block = blk[seq, at]
    pages = s["table"][seq, block].long()
    pos = block[:, None] * page + torch.arange(page, device="cuda")
    held = pos < s["old"][seq, None]
    row = pos - s["old"][seq, None]
    is_new = (row >= 0) & (row < n[seq, None])
    fresh = x.float()[(s["cu"][seq, None] + row).clamp(0, x.shape[0] - 1)].transpose(1, 2)     # [blocks, heads, page, dim]
    is_new, held = is_new[:, None, :, None], held[:, None, :, None]
    fresh = torch.where(is_new, fresh, 0.0)
    amax = torch.where(fresh.isfinite(), fresh.abs(), 0.0).amax(dim=(2, 3))
    m, e = torch.frexp(amax)                                  # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), E_MIN).clamp(E_MIN, E_MAX)
    was = scales[pages]
    scale = torch.ldexp(torch.ones_like(amax), e)
    scale = torch.where(held.any(2)[..., 0], torch.maximum(scale, was), scale)
    before = codes[pages]
    value = torch.where(held, before.view(torch.float8_e4m3fn).float() * was[..., None, None], fresh)
    q = (value / scale[..., None, None]).clamp(-448, 448)
    q = torch.where(value.isfinite(), q, math.nan).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[pages] = torch.where(held | is_new, q, before)
    scales[pages] = scale


def _plain_read(s, c, codes, scales):
    seq = torch.bucketize(torch.arange(s["back_total"], device="cuda"), s["back"][1:], right=True)
    pos = s["from"][seq] + torch.arange(s["back_total"], device="cuda") - s["back"][seq]
    pages = s["table"][seq, pos // c["page"]].long()
    x = codes.view(torch.float8_e4m3fn)[pages, :, pos % c["page"]].float()
    return (x * scales[pages][..., None]).bfloat16()


def _plain_attention(s, c):
    q, (kc, ks, vc, vs), page = s["q"], s["cache"], c["page"]
    batch, hk, dim, g = c["batch"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    most, length = s["most"], -(-s["kv_most"] // page) * page
    pages = s["table"][:, :length // page].long()
    k, v = [(x[pages].view(torch.float8_e4m3fn).float() * f[pages][..., None, None]).transpose(1, 2)
            .reshape(batch, hk, length, dim) for x, f in ((kc, ks), (vc, vs))]
    n = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(most, device="cuda")
    row = (s["cu"][:-1, None] + i).clamp(max=q.shape[0] - 1).long()
    x = q.float()[row].view(batch, most, hk, g, dim).permute(0, 2, 3, 1, 4).reshape(batch, hk, g * most, dim)
    pos = (s["kv"] - n)[:, None, None] + i[None, :, None]
    j = torch.arange(length, device="cuda")
    hidden = (j >= s["kv"][:, None, None]) | (pos < 0) & bool(c["causal"])
    if c["causal"]:
        hidden = hidden | (j > pos)
    if c["window"]:
        hidden = hidden | (j <= pos - c["window"])
    score = (x @ k.transpose(2, 3)).mul_(1 / math.sqrt(dim)).view(batch, hk, g, most, length)
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight.view(batch, hk, g * most, length) @ v).view(batch, hk, g, most, dim)
    out = torch.where(total > 0, out / total, 0.0)
    keep = i < n[:, None]
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, most, c["heads"], dim)[keep].bfloat16()
    if not c["lse"]:
        return {"out": out}
    return {"out": out, "lse": (top + total.log()).permute(0, 3, 1, 2, 4).reshape(batch, most, c["heads"])[keep]}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rope":
        return {"out": _rotate(s["x"], s["positions"], s["freqs"], s["dims"], c["layout"], c["inverse"])}
    if c["op"] == "attn":
        return _plain_attention(s, c)
    kc, ks, vc, vs = s["cache"]
    if c["op"] == "write":
        k = _rotate(s["k"], s["positions"], s["freqs"], s["dims"], 0, 0) if c["rope"] else s["k"]
        _plain_write(s, c, k, kc, ks)
        _plain_write(s, c, s["v"], vc, vs)
        if not c["read"]:
            return {"k": kc.view(torch.float8_e4m3fn), "k_scale": ks, "v": vc.view(torch.float8_e4m3fn), "v_scale": vs}
    return {"k": _plain_read(s, c, kc, ks), "v": _plain_read(s, c, vc, vs)}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import dit_modulate_absmax_gb300 as h3
    c = s["case"]
    if c["op"] == "rope":
        rope = h3.Rope(s["positions"], s["freqs"], s["dims"], layout=LAYOUTS[c["layout"]])
        return {"out": h3.rope_axes(s["x"], rope, inverse=bool(c["inverse"]))}
    cache = h3.KVCache(*s["cache"])
    if c["op"] == "attn":
        out, lse = h3.kv_attention(s["q"], cache, s["table"], s["kv"], s["cu"], s["most"], s["kv_most"],
                                   causal=bool(c["causal"]), window=c["window"], return_lse=bool(c["lse"]))
        return {"out": out, "lse": lse} if c["lse"] else {"out": out}
    if c["op"] == "write":
        rope = h3.Rope(s["positions"], s["freqs"], s["dims"]) if c["rope"] else None
        h3.kv_cache_write(cache, s["k"], s["v"], s["table"], s["old"], s["cu"], s["new"], rope=rope)
        if not c["read"]:
            return {"k": cache.k_codes.view(torch.float8_e4m3fn), "k_scale": cache.k_scale,
                    "v": cache.v_codes.view(torch.float8_e4m3fn), "v_scale": cache.v_scale}
    k, v = h3.kv_cache_read(cache, s["table"], s["from"], s["back"], s["back_total"], s["back_most"])
    return {"k": k, "v": v}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rope(x, positions, freqs, dims, layout, inverse):
    y, at, f = x.double(), 0, 0
    for a, d in enumerate(dims):
        phi = positions[:, a, None].double() * freqs[f:f + d // 2]
        z = torch.polar(torch.ones_like(phi), -phi if inverse else phi)[:, None]
        part = y[:, :, at:at + d]
        if layout == 0:
            part.copy_(torch.view_as_real(torch.view_as_complex(part.unflatten(2, (-1, 2)).contiguous()) * z).flatten(2))
        else:
            w = torch.complex(part[..., :d // 2].contiguous(), part[..., d // 2:].contiguous()) * z
            part.copy_(torch.cat([w.real, w.imag], 2))
        at, f = at + d, f + d // 2
    return y


def _exact_e4m3(x):
    """The nearest E4M3 value, ties to even, saturating."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_cache(s, c, x, codes, scales):
    """A sequence's blocks one after another; codes as the values they stand for, without their scale."""
    value, scales, page = codes.view(torch.float8_e4m3fn).double(), scales.double(), c["page"]
    cu, old, table = s["cu"].tolist(), s["old"].tolist(), s["table"].tolist()
    for b in range(c["batch"]):
        n = cu[b + 1] - cu[b]
        for blk in range(old[b] // page, (old[b] + n - 1) // page + 1):
            p, lo, hi = table[b][blk], max(blk * page, old[b]), min((blk + 1) * page, old[b] + n)
            held, new = lo - blk * page, x[cu[b] + lo - old[b]:cu[b] + hi - old[b]].double().transpose(0, 1)
            most = new.abs().amax(dim=(1, 2))
            need = (torch.floor(torch.log2(most)) - 8).exp2()
            need = torch.where(most > 448 * need, 2 * need, need).clamp(2.0 ** E_MIN, 2.0 ** E_MAX)
            scale = torch.maximum(need, scales[p]) if held else need
            value[p, :, :held] = _exact_e4m3(value[p, :, :held] * (scales[p] / scale)[:, None, None])
            value[p, :, held:held + hi - lo] = _exact_e4m3(new / scale[:, None, None])
            scales[p] = scale
    return value, scales


def _exact_attention(s, c):
    kc, ks, vc, vs = s["cache"]
    cu, kv, page, g = s["cu"].tolist(), s["kv"].tolist(), c["page"], c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        L, n = kv[b], cu[b + 1] - cu[b]
        ids = s["table"][b, :-(-L // page)].long()
        pos, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
        see = torch.ones(n, L, dtype=torch.bool, device="cuda")
        if c["causal"]:
            see &= j <= pos
        if c["window"]:
            see &= j > pos - c["window"]
        for h in range(c["kv_heads"]):
            k, v = [(x[ids, h].view(torch.float8_e4m3fn).double() * f[ids, h, None, None]).flatten(0, 1)[:L]
                    for x, f in ((kc, ks), (vc, vs))]
            for t in range(h * g, h * g + g):
                score = (s["q"][cu[b]:cu[b + 1], t].double() @ k.T / math.sqrt(c["dim"])).masked_fill_(~see, -math.inf)
                lse[cu[b]:cu[b + 1], t] = torch.logsumexp(score, 1)
                out[cu[b]:cu[b + 1], t] = torch.softmax(score, 1) @ v
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return {"out": _exact_rope(s["x"], s["positions"], s["freqs"], s["dims"], c["layout"], c["inverse"])}
    if c["op"] == "attn":
        if work(case)["flops"] > 8e12 or sum(_attn_lengths(c)[1]) * c["heads"] > 4e7:
            return None
        return _exact_attention(s, c)
    kc, ks, vc, vs = s["cache"]
    if c["op"] == "write":
        k = _exact_rope(s["k"], s["positions"], s["freqs"], s["dims"], 0, 0) if c["rope"] else s["k"]
        (kc, ks), (vc, vs) = _exact_cache(s, c, k, kc, ks), _exact_cache(s, c, s["v"], vc, vs)
        if not c["read"]:
            return {"k": kc, "k_scale": ks, "v": vc, "v_scale": vs}
        kc, vc = kc * ks[..., None, None], vc * vs[..., None, None]
    else:
        kc, vc = [x.view(torch.float8_e4m3fn).double() * f[..., None, None] for x, f in ((kc, ks), (vc, vs))]
    got, start, page = {"k": [], "v": []}, s["from"].tolist(), c["page"]
    back = s["back"].tolist()
    for b in range(c["batch"]):
        pos = torch.arange(start[b], start[b] + back[b + 1] - back[b], device="cuda")
        ids = s["table"][b, pos // page].long()
        got["k"].append(kc[ids, :, pos % page])
        got["v"].append(vc[ids, :, pos % page])
    return {n: torch.cat(x) for n, x in got.items()}
