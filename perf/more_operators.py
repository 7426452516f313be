"""Work over further operators of the attention path: per-head norms of queries
and keys with their rotation in the same pass (and the gradients), attention
with a sliding window whose first tokens stay visible, attention of sequences
that share a prefix, and the tables of a paged cache built from request lengths.

With ``own`` false every operator is computed in its plain form, elementary
torch operations in 32 bits (64 for angles and long sums) rounded once at the
end; with ``own`` true the same pass makes the calls a user makes of this
framework.  Sizes are those of the streaming DiT block (37,810 tokens, 5,042 a
chunk, 56 heads of 128, frames of 3,600 and 1,560 tokens) and generic ones for
token-by-token decoding.
"""
import math

import torch

own = False

EPS = 1e-6
LAYOUTS = ("interleaved", "halves")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decoding step's queries and keys of 32 requests (latency)
        dict(name="norm_decode", op="norm", tokens=32, hq=64, hk=8, dim=128, d0=128, d1=0, d2=0, layout=1, ld=80, wide=0,
             grad=0),
        # the whole video's queries and keys, read from the QKV projection's rows
        dict(name="norm_video", op="norm", tokens=37_810, hq=56, hk=56, dim=128, d0=44, d1=42, d2=42, layout=0, ld=168,
             wide=0, grad=0),
        # training: gradients of a chunk's queries and keys and of both weights
        dict(name="norm_grad_chunk", op="norm", tokens=5_042, hq=56, hk=56, dim=128, d0=44, d1=42, d2=42, layout=0, ld=168,
             wide=0, grad=1),
        # training on text: grouped heads of 64 channels, pairs split in halves, weights kept in 32 bits
        dict(name="norm_grad_text", op="norm", tokens=1_237, hq=20, hk=4, dim=64, d0=64, d1=0, d2=0, layout=1, ld=28, wide=1,
             grad=1),
        # a batch of 32 ragged requests decoding under a window, eight query heads to a key head
        dict(name="sink_decode_batch", op="sink", batch=32, q=1, kv=8_190, heads=64, kv_heads=8, dim=128, page=64, causal=1,
             window=2_000, sinks=64, lse=0),
        # one very long request decoding, four first tokens kept
        dict(name="sink_decode_long", op="sink", batch=1, q=1, kv=262_143, heads=32, kv_heads=8, dim=128, page=128, causal=1,
             window=65_536, sinks=4, lse=1),
        # a video chunk that sees the first frame, and the frames within its window
        dict(name="sink_chunk", op="sink", batch=1, q=5_042, kv=37_810, heads=56, kv_heads=56, dim=128, page=64, causal=0,
             window=16_384, sinks=3_600, lse=0),
        # a few requests behind a short instruction (latency)
        dict(name="shared_few", op="shared", groups=1, batch=3, q=1, prefix=777, kv=40, heads=16, kv_heads=4, dim=64, page=16,
             causal=1, lse=0),
        # 64 requests decoding behind one long document
        dict(name="shared_decode", op="shared", groups=1, batch=64, q=1, prefix=16_381, kv=500, heads=64, kv_heads=8, dim=128,
             page=64, causal=1, lse=1),
        # guided sampling: four samples behind each of two prompts, each denoising a frame's tokens over the frames so far
        dict(name="shared_samples", op="shared", groups=2, batch=8, q=1_560, prefix=4_680, kv=1_560, heads=56, kv_heads=56,
             dim=128, page=64, causal=0, lse=0),
        # the tables of a decoding step of 64 requests
        dict(name="tables_decode", op="tables", batch=64, new=1, old=8_190, page=64),
        # the tables of a thousand prompts, some of which hold tokens already
        dict(name="tables_prompts", op="tables", batch=1_000, new=503, old=260, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "sink", "sink", "shared", "shared", "tables"])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        dim = rng.choice([64, 96, 128, 128, 256])
        hq, hk, grad = rng.randint(1, 56), rng.randint(0, 28), rng.randint(0, 1)
        d1 = rng.choice([0, 2 * rng.randint(1, dim // 6)])
        d0 = dim - 2 * d1 - rng.choice([0, 0, 8])
        return dict(op=op, tokens=_log(rng, 1, 18_720), hq=hq, hk=hk, dim=dim, d0=d0, d1=d1, d2=d1, layout=rng.randint(0, 1),
                    ld=hq + hk + rng.randint(0, 28), wide=rng.randint(0, 1), grad=grad)
    if op == "tables":
        new = rng.choice([1, _log(rng, 1, 5_042)])
        return dict(op=op, batch=min(_log(rng, 1, 4_000), 1 + 300_000 // new), new=new, old=_log(rng, 1, 8_190) - 1, page=page)
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.randint(1, 8)
    group = rng.choice([1, 2, 4, 5, 8])
    q = rng.choice([1, 1, _log(rng, 2, 24), _log(rng, 2, 5_042)])
    batch = _log(rng, 1, 32) if q <= 24 else rng.randint(1, 4)
    fit = 4_000_000_000 // (batch * q * kv_heads * group)
    if op == "sink":
        kv = max(q, min(_log(rng, 16, 65_536), fit, 2_000_000 // batch))
        return dict(op=op, batch=batch, q=q, kv=kv, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page,
                    causal=rng.randint(0, 1), window=_log(rng, 1, 8_192), sinks=_log(rng, 1, 3_600), lse=rng.randint(0, 1))
    prefix = max(1, min(_log(rng, 16, 32_768), fit // 2, 1_000_000 // batch))
    kv = max(q, min(_log(rng, 1, 2_000), fit // 2))
    return dict(op=op, groups=rng.randint(1, min(3, batch)), batch=batch, q=q, prefix=prefix, kv=kv, heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim, page=page, causal=rng.randint(0, 1), lse=rng.randint(0, 1))


def _ragged(most, batch):
    """Lengths of a batch: the first is the longest, the others spread down to a quarter of it."""
    return [max(1, round(most * (1 - 0.75 * ((b * 0.6180339887498949) % 1.0)))) if most else 0 for b in range(batch)]


def _attn_lengths(c):
    qs = _ragged(c["q"], c["batch"])
    return qs, [max(k, n) for k, n in zip(_ragged(c["kv"], c["batch"]), qs)]


def _group_of(c):
    """Sequences of each prefix: contiguous, as even as they go."""
    return [b * c["groups"] // c["batch"] for b in range(c["batch"])]


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["tokens"] * (c["hq"] + c["hk"]) * c["dim"]
        axes = 4 * c["tokens"] * ((c["d0"] > 0) + (c["d1"] > 0) + (c["d2"] > 0))
        return {"bytes": (6 if c["grad"] else 4) * n + axes, "flops": (20 if c["grad"] else 8) * n}
    if c["op"] == "tables":
        new, old = _ragged(c["new"], c["batch"]), _ragged(c["old"], c["batch"])
        taken = sum(_pages(o + n, c["page"]) - _pages(o, c["page"]) for o, n in zip(old, new))
        return {"bytes": 12 * sum(new) + 8 * taken + 20 * c["batch"], "flops": 4 * sum(new)}
    qs, ks = _attn_lengths(c)
    pairs = keys = 0
    for n, L in zip(qs, ks):
        first = L - n                                              # position of the first query
        if c["op"] == "shared":
            pairs += sum(range(first + 1, L + 1)) if c["causal"] else n * L
            keys += L
            continue
        for pos in range(first, L):
            low = max(0, pos - c["window"] + 1)
            pairs += (pos + 1 if c["causal"] else L) - low + min(c["sinks"], low)
        low = max(0, first - c["window"] + 1)
        keys += L - low + min(c["sinks"], low)
    if c["op"] == "shared":
        pairs += sum(qs) * c["prefix"]
        keys += c["groups"] * c["prefix"]
    rows = sum(qs) * c["heads"] * c["dim"]
    return {"bytes": 4 * rows + 2 * keys * c["kv_heads"] * c["dim"] + (4 * sum(qs) * c["heads"] if c["lse"] else 0),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _positions(tokens, axes, gen):
    """Time, height and width of a video's tokens, 45 x 80 patches a frame, from a frame of the seed; or a text's."""
    i = torch.arange(tokens, device="cuda")
    if axes == 1:
        return (int(torch.randint(0, 100_000, (1,), generator=gen, device="cuda")) + i).float()[:, None]
    first = int(torch.randint(0, 32, (1,), generator=gen, device="cuda"))
    return torch.stack([first + i // 3600, i // 80 % 45, i % 80], dim=1).float()


def _frequencies(dims):
    """Radians per unit of position for each rotated pair, 10000^(-2j/d) along each axis."""
    return torch.cat([10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in dims]).cuda()


def _tables(lengths, page, ids):
    """Page tables over the page numbers given, one sequence after another; entries without a page are -1."""
    counts = [_pages(n, page) for n in lengths]
    table = torch.full((len(lengths), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    owner = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(counts))
    within = torch.arange(sum(counts)) - torch.tensor([0] + counts).cumsum(0)[owner]
    table[owner.cuda(), within.cuda()] = ids[:sum(counts)]
    return table, sum(counts)


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


def _ints(values):
    return torch.tensor(values, device="cuda").int()


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
    if c["op"] == "norm":
        dims = tuple(d for d in (c["d0"], c["d1"], c["d2"]) if d)
        rows = _bf16((c["tokens"], c["ld"], c["dim"]), gen, 1.7)          # of a QKV projection
        heads = {"q": rows[:, :c["hq"]], "k": rows[:, c["hq"]:c["hq"] + c["hk"]] if c["hk"] else None}
        kind = torch.float32 if c["wide"] else torch.bfloat16
        weight = [(1 + 0.25 * torch.randn(c["dim"], generator=gen, device="cuda")).to(kind) for _ in "qk"]
        s |= {"heads": heads, "weight": {"q": weight[0], "k": weight[1] if c["hk"] else None},
              "positions": _positions(c["tokens"], len(dims), gen), "freqs": _frequencies(dims), "dims": dims}
        if c["grad"]:
            s["dy"] = {n: None if x is None else _bf16(x.shape, gen, 0.01) for n, x in heads.items()}
        return s
    if c["op"] == "tables":
        new, old = _ragged(c["new"], c["batch"]), _ragged(c["old"], c["batch"])
        pages = sum(_pages(o + n, c["page"]) for o, n in zip(old, new)) + 5
        ids = torch.randperm(pages, generator=gen, device="cuda").int()
        table, used = _tables(old, c["page"], ids)
        room = max(_pages(o + n, c["page"]) for o, n in zip(old, new)) + 1
        table = torch.cat([table, table.new_full((c["batch"], room), -1)], 1)[:, :room].contiguous()
        return s | {"held": _ints(old), "new": _ints(new), "table": table, "free": ids[used:].contiguous(), "free_at": _ints([2]),
                    "tokens": sum(new) + 7, "most": max(new), "pages": pages}
    qs, ks = _attn_lengths(c)
    shared = [c["prefix"]] * c["groups"] if c["op"] == "shared" else []
    total = sum(_pages(n, c["page"]) for n in ks + shared) + 3
    ids = torch.randperm(total, generator=gen, device="cuda").int()
    table, used = _tables(ks, c["page"], ids)
    s |= {"q": _bf16((sum(qs), c["heads"], c["dim"]), gen, 2.0), "table": table, "cu": _cu(qs), "most": max(qs),
          "cache": _filled(total, c["kv_heads"], c["page"], c["dim"], gen), "kv": _ints(ks), "kv_most": max(ks)}
    if shared:
        of = _group_of(c)
        rows = [sum(n for n, g in zip(qs, of) if g == i) for i in range(c["groups"])]
        s |= {"p_table": _tables(shared, c["page"], ids[used:])[0], "p_len": _ints(shared), "p_cu": _cu(rows),
              "p_most": max(rows), "p_of": torch.tensor(of, device="cuda")}
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _rotate(x, s, layout, inverse):
    """x [tokens, heads, dim] in 32 bits, rotated pair by pair."""
    dims, at, y = s["dims"], 0, x.clone()
    for a, d in enumerate(dims):
        j = torch.arange(d // 2, device="cuda")
        lo = at + (2 * j if layout == 0 else j)
        hi = lo + (1 if layout == 0 else d // 2)
        angle = s["positions"][:, a, None].double() * s["freqs"][at // 2:(at + d) // 2]
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None] * (-1 if inverse else 1)
        y[:, :, lo] = x[:, :, lo] * cos - x[:, :, hi] * sin
        y[:, :, hi] = x[:, :, lo] * sin + x[:, :, hi] * cos
        at += d
    return y


def _plain_norm(s, c):
    out = {}
    for n, x in s["heads"].items():
        if x is None:
            continue
        w, x = s["weight"][n].float(), x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if not c["grad"]:
            out[n] = _rotate(x * r * w, s, c["layout"], False).bfloat16()
            continue
        g = _rotate(s["dy"][n].float(), s, c["layout"], True)
        hat = x * r
        out["d" + n] = (r * (w * g - hat * (w * g * hat).mean(-1, keepdim=True))).bfloat16()
        out[f"d{n}_weight"] = (g * hat).sum((0, 1), dtype=torch.float64).float()
    return out


def _keys_of(s, c, table, length):
    """Keys and values [batch, kv_heads, length, dim] of the tables' rows, in 32 bits."""
    kc, ks, vc, vs = s["cache"]
    pages = table[:, :length // c["page"]].clamp(min=0).long()
    return [(x[pages].view(torch.float8_e4m3fn).float() * f[pages][..., None, None]).transpose(1, 2)
            .reshape(len(table), c["kv_heads"], length, c["dim"]) for x, f in ((kc, ks), (vc, vs))]


def _plain_attention(s, c):
    q, page = s["q"], c["page"]
    batch, hk, dim, g = c["batch"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    most, length = s["most"], _pages(s["kv_most"], page) * page
    k, v = _keys_of(s, c, s["table"], length)
    n = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(most, device="cuda")
    row = (s["cu"][:-1, None] + i).clamp(max=q.shape[0] - 1).long()
    x = q.float()[row].view(batch, most, hk, g, dim).permute(0, 2, 3, 1, 4).reshape(batch, hk, g * most, dim)
    pos = (s["kv"] - n)[:, None, None] + i[None, :, None]
    j = torch.arange(length, device="cuda")
    hidden = (j >= s["kv"][:, None, None]).expand(batch, most, length)
    if c["causal"]:
        hidden = hidden | (j > pos)
    if c["op"] == "sink":
        hidden = hidden | (j <= pos - c["window"]) & (j >= c["sinks"])
    else:                                                          # the prefix comes before all of it, and is seen by all
        before = _pages(c["prefix"], page) * page
        pk, pv = _keys_of(s, c, s["p_table"], before)
        k, v = torch.cat([pk[s["p_of"]], k], 2), torch.cat([pv[s["p_of"]], v], 2)
        past = (torch.arange(before, device="cuda") >= s["p_len"][s["p_of"], None])[:, None].expand(batch, most, before)
        hidden = torch.cat([past, hidden], 2)
    score = (x @ k.transpose(2, 3)).mul_(1 / math.sqrt(dim)).view(batch, hk, g, most, -1)
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight.view(batch, hk, g * most, -1) @ v).view(batch, hk, g, most, dim)
    out = torch.where(total > 0, out / total, 0.0)
    keep = i < n[:, None]
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, most, c["heads"], dim)[keep].bfloat16()
    if not c["lse"]:
        return {"out": out}
    return {"out": out, "lse": (top + total.log()).permute(0, 3, 1, 2, 4).reshape(batch, most, c["heads"])[keep]}


def _plain_tables(s, c):
    held, new, table, page = s["held"], s["new"], s["table"], c["page"]
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)]).int()
    kv = held + new
    first, last = (held + page - 1) // page, (kv + page - 1) // page
    before = torch.cat([first.new_zeros(1), (last - first).cumsum(0)])
    p = torch.arange(table.shape[1], device="cuda")
    fresh = (p >= first[:, None]) & (p < last[:, None])
    take = s["free_at"] + before[:-1, None] + p - first[:, None]
    table[fresh] = s["free"][take[fresh].long()]
    i = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(cu[1:], i, right=True).clamp(max=c["batch"] - 1)
    pos = held[seq] + i - cu[seq]
    real = i < cu[-1]
    at = torch.where(real, pos // page, 0)
    slots = torch.where(real, table[seq, at].long() * page + pos % page, -1)
    return {"cu_tokens": cu, "kv_len": kv, "slots": slots, "positions": torch.where(real, pos, -1).float(), "page_table": table,
            "free_at": (s["free_at"] + before[-1]).int()}


def _run_plain(s):
    c = s["case"]
    return {"norm": _plain_norm, "sink": _plain_attention, "shared": _plain_attention, "tables": _plain_tables}[c["op"]](s, c)


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import dit_modulate_absmax_gb300 as h3
    c = s["case"]
    if c["op"] == "norm":
        rope = h3.Rope(s["positions"], s["freqs"], s["dims"], layout=LAYOUTS[c["layout"]])
        x, w = s["heads"], s["weight"]
        if not c["grad"]:
            q, k = h3.norm_rope(x["q"], x["k"], q_weight=w["q"], k_weight=w["k"], rope=rope, eps=EPS)
            return {"q": q} if k is None else {"q": q, "k": k}
        dq, dk, dqw, dkw = h3.norm_rope_backward(s["dy"]["q"], s["dy"]["k"], x["q"], x["k"], q_weight=w["q"], k_weight=w["k"],
                                                 rope=rope, eps=EPS)
        out = {"dq": dq, "dq_weight": dqw}
        return out if dk is None else out | {"dk": dk, "dk_weight": dkw}
    if c["op"] == "tables":
        t = h3.kv_tables(s["held"], s["new"], s["table"], s["free"], s["free_at"], c["page"], s["pages"], s["tokens"], s["most"])
        return {"cu_tokens": t.cu_tokens, "kv_len": t.kv_len, "slots": t.slots, "positions": t.positions,
                "page_table": s["table"], "free_at": t.free_at}
    cache = h3.KVCache(*s["cache"])
    if c["op"] == "sink":
        out, lse = h3.kv_attention(s["q"], cache, s["table"], s["kv"], s["cu"], s["most"], s["kv_most"],
                                   causal=bool(c["causal"]), window=c["window"], sinks=c["sinks"], return_lse=bool(c["lse"]))
    else:
        prefix = h3.SharedPrefix(s["p_table"], s["p_len"], s["p_cu"], s["p_most"], c["prefix"])
        out, lse = h3.kv_attention_shared(s["q"], cache, prefix, s["table"], s["kv"], s["cu"], s["most"], s["kv_most"],
                                          causal=bool(c["causal"]), return_lse=bool(c["lse"]))
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _turns(s):
    """The rotation of each token as unit complex numbers, one row of pairs an axis."""
    f, out = 0, []
    for a, d in enumerate(s["dims"]):
        phi = s["positions"][:, a, None].double() * s["freqs"][f:f + d // 2]
        out.append(torch.polar(torch.ones_like(phi), phi)[:, None])
        f += d // 2
    return out


def _exact_turn(x, s, layout, back):
    at, parts = 0, []
    for z in _turns(s):
        d = 2 * z.shape[2]
        part, z = x[:, :, at:at + d], z.conj() if back else z
        if layout == 0:
            parts.append(torch.view_as_real(torch.view_as_complex(part.unflatten(2, (-1, 2)).contiguous()) * z).flatten(2))
        else:
            w = torch.complex(part[..., :d // 2].contiguous(), part[..., d // 2:].contiguous()) * z
            parts.append(torch.cat([w.real, w.imag], 2))
        at += d
    return torch.cat(parts + [x[:, :, at:]], 2)


def _exact_norm(s, c):
    out = {}
    for n, x in s["heads"].items():
        if x is None:
            continue
        x, w = x.double(), s["weight"][n].double()
        size = torch.sqrt(x.square().sum(2, keepdim=True) / c["dim"] + EPS)
        if not c["grad"]:
            out[n] = _exact_turn(x / size * w, s, c["layout"], False)
            continue
        g = _exact_turn(s["dy"][n].double(), s, c["layout"], True)
        along = torch.einsum("thd,thd,d->th", g, x, w)[..., None] / c["dim"]
        out["d" + n] = g * w / size - x * along / size ** 3
        out[f"d{n}_weight"] = torch.einsum("thd,thd->d", g, x / size)
    return out


def _exact_attention(s, c):
    kc, ks, vc, vs = s["cache"]
    cu, kv, page, g = s["cu"].tolist(), s["kv"].tolist(), c["page"], c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        L, n, before = kv[b], cu[b + 1] - cu[b], 0
        ids, at = s["table"][b, :_pages(L, page)].long(), torch.arange(L, device="cuda")
        if c["op"] == "shared":
            before = c["prefix"]
            mine = s["p_table"][int(s["p_of"][b]), :_pages(before, page)].long()
            at = torch.cat([torch.arange(before, device="cuda"), len(mine) * page + at])
            ids = torch.cat([mine, ids])
        pos, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(-before, L, device="cuda")
        see = torch.ones(n, before + L, dtype=torch.bool, device="cuda")
        if c["causal"]:
            see &= j <= pos
        if c["op"] == "sink":
            see &= (j > pos - c["window"]) | (j < c["sinks"])
        for h in range(c["kv_heads"]):
            k, v = [(x[ids, h].view(torch.float8_e4m3fn).double() * f[ids, h, None, None]).flatten(0, 1)[at]
                    for x, f in ((kc, ks), (vc, vs))]
            for t in range(h * g, h * g + g):
                score = (s["q"][cu[b]:cu[b + 1], t].double() @ k.T / math.sqrt(c["dim"])).masked_fill_(~see, -math.inf)
                lse[cu[b]:cu[b + 1], t] = torch.logsumexp(score, 1)
                out[cu[b]:cu[b + 1], t] = torch.softmax(score, 1) @ v
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _exact_tables(s, c):
    """One sequence after another, on the host."""
    held, new, table, free, page = s["held"].tolist(), s["new"].tolist(), s["table"].tolist(), s["free"].tolist(), c["page"]
    cu, kv, slots, positions, at = [0], [], [], [], s["free_at"].tolist()[0]
    for b in range(c["batch"]):
        for pos in range(held[b], held[b] + new[b]):
            if pos % page == 0:
                table[b][pos // page] = free[at]
                at += 1
            slots.append(table[b][pos // page] * page + pos % page)
            positions.append(float(pos))
        cu.append(cu[-1] + new[b])
        kv.append(held[b] + new[b])
    behind = [-1] * (s["tokens"] - len(slots))
    return {"cu_tokens": _ints(cu), "kv_len": _ints(kv), "slots": torch.tensor(slots + behind, device="cuda"),
            "positions": torch.tensor(positions + [float(x) for x in behind], device="cuda"), "page_table": _ints(table),
            "free_at": _ints([at])}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        return _exact_norm(s, c)
    if c["op"] == "tables":
        return _exact_tables(s, c)
    if work(case)["flops"] > 8e12 or sum(_attn_lengths(c)[1]) * c["heads"] > 4e7:
        return None
    return _exact_attention(s, c)
