"""What is measured of the attention side of a block: rotary positions, a
paged key/value cache held in 4 bits (append, read), the attention that reads
it, and eviction from it by accumulated attention weight.

A case names an operator ("op") and its sizes and types; prepare() makes its
inputs from a seed, run() is one pass (plain torch operations, or this
package's kernels where `own` is true), work() the bytes and operations that
a pass cannot do without, exact() the result in 64 bits.

The cache: codes [pages, kv heads, page size, D / 2] bytes of two's-complement
nibbles (the low one is the even column), scales bfloat16 [pages, kv heads,
D / 64, page size], one per 64 columns of a row; value = code * scale.  Row r
of a sequence stands in page table[s, r // page size] at r % page size.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
GROUP = 64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    rot, app, att, evi = {"op": "rotary"}, {"op": "append"}, {"op": "attention"}, {"op": "evict"}
    return [
        # queries and keys of one decoded token, as one view of the fused projection: latency alone
        dict(rot, name="rotary one token", tokens=1, heads=72, dim=128, part=128, type="bf16", interleaved=False,
             far=4096, scale=1.0, inverse=False),
        # a prompt deep in a long context, half of each head, interleaved pairs
        dict(rot, name="rotary prompt", tokens=4096, heads=56, dim=128, part=64, type="f16", interleaved=True,
             far=1000000, scale=1.25, inverse=False),
        # one new token of each sequence of a decode batch
        dict(app, name="append decode", seqs=64, new=1, heads=8, dim=128, page=64, type="bf16", past=2048),
        # ragged prompts, small pages
        dict(app, name="append prompts", seqs=3, new=2000, heads=4, dim=256, page=16, type="f16", past=500),
        # the first tokens of one conversation: latency alone
        dict(att, name="attention one short", seqs=1, new=1, q_heads=64, heads=8, dim=128, page=64, length=517,
             type="bf16", window=0, weights=False),
        # a decode batch of ragged contexts
        dict(att, name="attention batch", seqs=64, new=1, q_heads=64, heads=8, dim=128, page=64, length=8192,
             type="bf16", window=0, weights=False),
        # one conversation with a long context
        dict(att, name="attention one long", seqs=1, new=1, q_heads=64, heads=8, dim=128, page=256, length=131071,
             type="bf16", window=0, weights=False),
        # a few drafted tokens of each sequence verified at once, in a window, a key head for every query head
        dict(att, name="attention drafts", seqs=16, new=5, q_heads=16, heads=16, dim=64, page=16, length=4000,
             type="f16", window=1024, weights=False),
        # a decode batch that also gathers the weights its eviction goes by
        dict(att, name="attention weights", seqs=16, new=1, q_heads=48, heads=8, dim=128, page=64, length=4096,
             type="bf16", window=0, weights=True),
        # pieces of two prompts on what is cached of them
        dict(att, name="attention prompts", seqs=2, new=1500, q_heads=64, heads=8, dim=128, page=64, length=16384,
             type="bf16", window=0, weights=False),
        # one conversation cut to half: latency
        dict(evi, name="evict one", seqs=1, heads=8, dim=128, page=64, length=600, keep=256),
        # a whole batch cut to half
        dict(evi, name="evict batch", seqs=16, heads=8, dim=128, page=64, length=8192, keep=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention", "evict"])
    dim, page = rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128, 256])
    if op == "rotary":
        dim = 2 * rng.randint(16, 128)
        heads = _log(rng, 1, 80)
        tokens = min(_log(rng, 1, 16384), 4096 * 56 * 64 // (heads * dim))
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "part": 2 * rng.randint(1, dim // 2),
                "type": rng.choice(["f32", "bf16", "f16"]), "interleaved": rng.random() < 0.5,
                "far": _log(rng, 1024, 4000000), "scale": rng.choice([1.0, 1.25]), "inverse": rng.random() < 0.5}
    if op == "append":
        heads, seqs = _log(rng, 1, 16), _log(rng, 1, 64)
        new = min(_log(rng, 1, 2048), 2 * 2000 * 4 * 256 // (seqs * heads * dim))
        return {"op": op, "seqs": seqs, "new": new, "heads": heads, "dim": dim, "page": page,
                "type": rng.choice(["f32", "bf16", "f16"]), "past": _log(rng, 1, 1024)}
    if op == "evict":
        heads = _log(rng, 1, 16)
        length = min(_log(rng, 64, 32768), 12 * 8 * 128 * 4096 // (heads * dim))
        seqs = min(_log(rng, 1, 32), 12 * 8 * 128 * 4096 // (heads * dim * length))
        return {"op": op, "seqs": seqs, "heads": heads, "dim": dim, "page": page, "length": length,
                "keep": max(1, int(length * rng.uniform(0.2, 0.9)))}
    heads, group = _log(rng, 1, 16), rng.choice([1, 2, 4, 6, 8, 16])
    group = min(group, 64 // heads)
    new = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
    # no more products and no more of the cache than the largest listed cases
    products, cached = 1500 * 16384 * 64 * 128, 40 * 8 * 128 * 4096
    length = max(new, min(_log(rng, 16, 65536), products // (new * heads * group * dim)))
    rows = new * heads * group * dim
    seqs = max(1, min(_log(rng, 1, 64), cached // (length * heads * dim), products // (length * rows), (30 << 20) // rows))
    return {"op": op, "seqs": seqs, "new": new, "q_heads": heads * group, "heads": heads, "dim": dim,
            "page": page, "length": length, "type": rng.choice(["bf16", "f16"]),
            "window": rng.choice([0, 0, _log(rng, 16, 8192)]), "weights": rng.random() < 0.3}


def _ragged(case):
    """(new tokens, lengths) of the case's sequences: new tokens up to `new`, lengths up to `length`, the first the
    largest.  Sizes belong to the case, not to the seed of its values."""
    c, rng = case, random.Random(case["seqs"] * 1000003 + case.get("new", 0) * 1009 + case.get("length", 0))
    if c["op"] == "evict":
        return None, [c["length"]] + [rng.randint(max(1, c["length"] // 3), c["length"]) for _ in range(c["seqs"] - 1)]
    n = [c["new"]] + [rng.randint(max(1, c["new"] // 3), c["new"]) for _ in range(c["seqs"] - 1)]
    if c["op"] == "append":
        return n, [m + rng.randint(0, c["past"]) for m in n]
    low = max(1, c["length"] // 8)
    return n, [c["length"]] + [max(m, rng.randint(low, c["length"])) for m in n[1:]]


def _pairs(n, length, window):
    """Pairs of a query and a key it sees, and the keys that any query sees."""
    seen = [min(p + 1, window or p + 1) for p in range(length - n, length)]
    return sum(seen), min(length, n + (window or length) - 1)


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["tokens"] * c["heads"]
        return {"bytes": 2 * n * c["dim"] * SIZE[c["type"]] + 8 * c["tokens"] + 2 * c["part"], "flops": 3 * n * c["part"]}
    row = c["heads"] * (c["dim"] + 4 * (c["dim"] // GROUP))  # a token's keys and values with their scales
    n, lengths = _ragged(c)
    if c["op"] == "append":
        # rows in, codes and scales out, and the same read back as float32 values
        return {"bytes": sum(n) * (2 * c["heads"] * c["dim"] * (SIZE[c["type"]] + 4) + 2 * row),
                "flops": sum(n) * 8 * c["heads"] * c["dim"]}
    if c["op"] == "evict":
        # every weight once, what is kept read and written, and read back as half precision values
        kept = [min(m, c["keep"]) for m in lengths]
        return {"bytes": sum(lengths) * 4 * c["heads"] + sum(kept) * (3 * row + 8 * c["heads"] + 4 * c["heads"] * c["dim"]),
                "flops": sum(lengths) * 8 * c["heads"]}
    pairs, keys = zip(*(_pairs(a, b, c["window"]) for a, b in zip(n, lengths)))
    b = sum(keys) * row + 4 * sum(n) * c["q_heads"] * c["dim"]
    if c["weights"]:
        b += sum(keys) * 8 * c["heads"]
    return {"bytes": b, "flops": 4 * sum(pairs) * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _codes(pages, heads, page, dim, g, dev):
    """Codes and scales as rows of normal values with a size for each channel quantise to."""
    gain = torch.exp(0.4 * torch.randn(heads, 1, dim, generator=g, device=dev))
    gain *= 2.4 / gain.square().mean(2, keepdim=True).sqrt()
    q = torch.randn(pages, heads, page, dim, generator=g, device=dev).mul_(gain).round_().clamp_(-7, 7).to(torch.int8)
    s = 0.4 * torch.exp(0.2 * torch.randn(pages, heads, dim // GROUP, page, generator=g, device=dev))
    q &= 15
    return q[..., 0::2].bitwise_or(q[..., 1::2] << 4).view(torch.uint8), s.to(torch.bfloat16)


def _pool(c, lengths, spare, g, dev):
    """Cache and table for sequences of these lengths, pages in no order; `spare` more rows for each sequence in a
    second table."""
    ps, S = c["page"], c["seqs"]
    width, more = -(-max(lengths) // ps), -(-spare // ps)
    pages = S * (width + more) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    st = dict(table=order[: S * width].view(S, width), lengths=torch.tensor(lengths, dtype=torch.int32, device=dev))
    st["k_codes"], st["k_scales"] = _codes(pages, c["heads"], ps, c["dim"], g, dev)
    st["v_codes"], st["v_scales"] = _codes(pages, c["heads"], ps, c["dim"], g, dev)
    if spare:
        st["into"] = order[S * width: S * (width + more)].view(S, more)
    return st


def prepare(case, seed, dev="cuda"):
    c = case
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if c["op"] == "rotary":
        # a view of the fused projection (the values' heads stand behind), positions up to `far`
        x = rnd(c["tokens"], c["heads"] + 8, c["dim"]).to(TYPES[c["type"]])[:, : c["heads"]]
        start = torch.randint(0, c["far"], (1,), generator=g, device=dev)
        pos = (start + torch.arange(c["tokens"], device=dev)).to(torch.int32)
        half = torch.arange(c["part"] // 2, device=dev, dtype=torch.float64)
        freq = (10000.0 ** (-2 * half / c["part"])).float()
        return dict(case=c, x=x, pos=pos, freq=freq, out=torch.empty_like(x, memory_format=torch.contiguous_format))
    n, lengths = _ragged(c)
    st = _pool(c, lengths, c["keep"] if c["op"] == "evict" else 0, g, dev)
    st["case"] = c
    if c["op"] == "evict":
        # what accumulates in use: heavy tails, the first tokens far ahead; the kept rows' places, read back below
        w = torch.exp(2 * rnd(*st["k_scales"].shape[:2], c["page"])) / c["length"]
        w[st["table"][:, 0].long(), :, :4] += 1
        st["weights"] = w
        st["read"] = torch.arange(c["seqs"] + 1, device=dev, dtype=torch.int32) * c["keep"]
        return st
    T = sum(n)
    st["offsets"] = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev)
    st["tokens"], st["most"] = T, max(n)
    if c["op"] == "append":
        # keys of different sizes by token and channel, as views of a fused projection
        kv = rnd(T, 2 * c["heads"], c["dim"]) * torch.exp(0.5 * rnd(T, 1, 1)) * torch.exp(0.5 * rnd(1, 1, c["dim"]))
        kv = kv.to(TYPES[c["type"]])
        st["k"], st["v"] = kv[:, : c["heads"]], kv[:, c["heads"]:]
        return st
    st["q"] = rnd(T, c["q_heads"] + 2 * c["heads"], c["dim"]).to(TYPES[c["type"]])[:, : c["q_heads"]]
    if c["weights"]:
        st["weights"] = torch.rand(st["k_scales"].shape[0], c["heads"], c["page"], generator=g, device=dev)
        st["sums"] = st["weights"].clone()
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _token_rows(st, c):
    """(sequence, row in its sequence, page, place in the page) of every new token."""
    t = torch.arange(st["tokens"], device=st["table"].device)
    off = st["offsets"].long()
    seq = torch.searchsorted(off[1:].contiguous(), t, right=True)
    row = st["lengths"].long()[seq] - off[seq + 1] + t
    return seq, row, st["table"].long()[seq, row // c["page"]], row % c["page"]


def _all_rows(table, rows, page):
    """(page, place) of the first `rows` rows of every sequence."""
    r = torch.arange(rows, device=table.device)
    return table.long()[:, r // page], (r % page).expand(table.shape[0], -1)


def _values(codes, scales, pages, places, dtype):
    """Values [..., kv heads, D] of the rows at (pages, places)."""
    b = codes[pages, :, places].view(torch.int8)
    q = torch.stack([(b << 4) >> 4, b >> 4], -1).flatten(-2).to(dtype)  # arithmetic shifts: the nibbles' signs
    s = scales[pages, :, :, places].to(dtype)
    return (q.unflatten(-1, (-1, GROUP)) * s.unsqueeze(-1)).flatten(-2)


def _quantise(x):
    """Codes (packed) and scales of rows x [T, heads, D], in 64 bits since codes sit next to borders."""
    v = x.double().unflatten(-1, (-1, GROUP))
    s = (v.abs().amax(-1) / 7).float().to(torch.bfloat16)
    q = torch.where(s.unsqueeze(-1) > 0, v / s.double().unsqueeze(-1), torch.zeros_like(v))
    q = q.round().clamp(-7, 7).to(torch.int8).flatten(-2) & 15
    return q[..., 0::2].bitwise_or(q[..., 1::2] << 4).view(torch.uint8), s


def _rotate(x, pos, freq, c, dtype):
    a = pos.double()[:, None] * freq.double()
    a = -a if c["inverse"] else a
    cos, sin = (c["scale"] * torch.cos(a)).to(dtype)[:, None], (c["scale"] * torch.sin(a)).to(dtype)[:, None]
    v, R = x.to(dtype), c["part"]
    a, b = (v[..., 0:R:2], v[..., 1:R:2]) if c["interleaved"] else (v[..., : R // 2], v[..., R // 2: R])
    p, q = a * cos - b * sin, a * sin + b * cos
    return torch.cat([torch.stack([p, q], -1).flatten(-2) if c["interleaved"] else torch.cat([p, q], -1), v[..., R:]], -1)


def _attention(st, c, dtype):
    """(outputs [T, q heads, D], weights per key [S, kv heads, rows]) with sequences padded to the longest."""
    S, K, G, D = c["seqs"], c["heads"], c["q_heads"] // c["heads"], c["dim"]
    N, L = st["most"], int(c["length"])
    dev = st["q"].device
    seq, row, _, _ = _token_rows(st, c)
    i = torch.arange(st["tokens"], device=dev) - st["offsets"].long()[seq]
    q = torch.zeros(S, N, K, G, D, dtype=dtype, device=dev)
    q[seq, i] = st["q"].to(dtype).unflatten(1, (K, G))
    at = torch.full((S, N), -1, device=dev)  # a padded query sees nothing
    at[seq, i] = row
    pages, places = _all_rows(st["table"], L, c["page"])
    k = _values(st["k_codes"], st["k_scales"], pages, places, dtype).permute(0, 2, 3, 1)
    s = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(S, K, N * G, D), k.contiguous()).mul_(D ** -0.5)
    del k
    key = torch.arange(L, device=dev)
    seen = key <= at[..., None]
    if c["window"]:
        seen &= key > at[..., None] - c["window"]
    s = s.view(S, K, N, G, L).masked_fill_(~seen[:, None, :, None], float("-inf"))
    s.sub_(torch.nan_to_num(s.amax(-1, keepdim=True), neginf=0.0)).exp_()
    s.div_(s.sum(-1, keepdim=True).clamp_min_(1e-30))
    w = s.sum((2, 3)) if c["weights"] else None
    v = _values(st["v_codes"], st["v_scales"], pages, places, dtype).transpose(1, 2).contiguous()
    o = torch.matmul(s.view(S, K, N * G, L), v).view(S, K, N, G, D).permute(0, 2, 1, 3, 4)[seq, i]
    return o.reshape(st["tokens"], c["q_heads"], D), w


def _first(c):
    return min(4, c["keep"] // 4)


def _recent(c):
    return c["keep"] // 4


def run(state):
    st, c = state, state["case"]
    if own:
        import routed_expert_ffn_f32_amd as cm
        if c["op"] == "rotary":
            return cm.rotary(st["x"], st["pos"], st["freq"], interleaved=c["interleaved"], scale=c["scale"],
                             inverse=c["inverse"], out=st["out"])
        if "cache" not in st:  # the handle that a program makes once
            st["cache"] = cm.KVCache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st.get("weights"))
        cache = st["cache"]
        if c["op"] == "append":
            cache.append(st["k"], st["v"], st["table"], st["lengths"], st["offsets"])
            return cache.read(st["tokens"], st["table"], st["lengths"], st["offsets"], dtype=torch.float32)
        if c["op"] == "evict":
            kept, lengths = cache.evict(c["keep"], st["table"], st["lengths"], st["into"], first=_first(c),
                                        recent=_recent(c))
            k, v = cache.read(c["seqs"] * c["keep"], st["into"], lengths, st["read"], dtype=torch.float16)
            return kept, lengths, k, v, st["weights"]
        offsets = None if c["new"] == 1 else st["offsets"]
        if c["weights"]:
            o = cache.attention(st["q"], st["table"], st["lengths"], offsets, window=c["window"],
                                weights_out=st["sums"])
            return o, st["sums"]
        return cache.attention(st["q"], st["table"], st["lengths"], offsets, window=c["window"])
    if c["op"] == "rotary":
        st["out"].copy_(_rotate(st["x"], st["pos"], st["freq"], c, torch.float32))
        return st["out"]
    if c["op"] == "append":
        _, _, page, place = _token_rows(st, c)
        for name in ("k", "v"):
            q, s = _quantise(st[name])
            st[name + "_codes"][page, :, place] = q
            st[name + "_scales"][page, :, :, place] = s
        return tuple(_values(st[name + "_codes"], st[name + "_scales"], page, place, torch.float32) for name in "kv")
    if c["op"] == "evict":
        return _evict(st, c)
    o, w = _attention(st, c, torch.float32)
    o = o.to(TYPES[c["type"]])
    if w is None:
        return o
    pages, places = _all_rows(st["table"], int(c["length"]), c["page"])
    inside = torch.arange(int(c["length"]), device=w.device) < st["lengths"].long()[:, None]
    pages, places = pages[inside], places[inside]
    st["sums"][pages, :, places] = st["weights"][pages, :, places] + w.transpose(1, 2)[inside]
    return o, st["sums"]


def _evict(st, c):
    """(kept rows [S, kv heads, keep], new lengths, values, weights): the first, the recent and the heaviest rows, in
    their order, copied to the pages of `into`."""
    S, K, keep, L = c["seqs"], c["heads"], c["keep"], c["length"]
    dev = st["table"].device
    length = st["lengths"].long()[:, None, None]
    pages, places = _all_rows(st["table"], L, c["page"])
    w = st["weights"][pages, :, places].transpose(1, 2)
    row = torch.arange(L, device=dev)
    always = (row < _first(c)) | (row >= length - _recent(c))
    rank = torch.where(always, torch.full_like(w, float("inf")), w)
    rank = torch.where(row < length, rank, torch.full_like(w, float("-inf")))
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(torch.arange(keep, device=dev) < length, best, L)
    kept = torch.sort(best, dim=-1).values
    new = st["lengths"].clamp_max(keep)
    inside = kept < L
    s, h, i = torch.nonzero(inside, as_tuple=True)
    at = kept[inside]
    src, sp = st["table"].long()[s, at // c["page"]], at % c["page"]
    dst, dp = st["into"].long()[s, i // c["page"]], i % c["page"]
    for name in ("k", "v"):
        st[name + "_codes"][dst, h, dp] = st[name + "_codes"][src, h, sp]
        st[name + "_scales"][dst, h, :, dp] = st[name + "_scales"][src, h, :, sp]
    st["weights"][dst, h, dp] = st["weights"][src, h, sp]
    pages, places = _all_rows(st["into"], keep, c["page"])
    # rows that read() gives: the last `keep` of every sequence, zeros before its first
    r = torch.arange(keep, device=dev) - keep + new.long()[:, None]
    pages, places = pages.gather(1, r.clamp_min(0)), places.gather(1, r.clamp_min(0))
    zero = (r < 0)[..., None, None]
    k, v = (_values(st[n + "_codes"], st[n + "_scales"], pages, places, torch.float32).masked_fill(zero, 0.0)
            .to(torch.float16).flatten(0, 1) for n in "kv")
    return torch.where(inside, kept, -1).to(torch.int32), new, k, v, st["weights"]


# ---------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _row_values(codes, scales, page, place):
    """float64 values [rows, kv heads, D] at (page, place), nibble by nibble."""
    b = codes[page, :, place].to(torch.int64)
    out = torch.empty(*b.shape[:2], 2 * b.shape[2], dtype=torch.float64, device=b.device)
    for i, nib in enumerate((b % 16, b // 16)):
        out[..., i::2] = torch.where(nib > 7, nib - 16, nib).double()
    return out * scales[page, :, :, place].double().repeat_interleave(GROUP, -1)


def exact(case, seed, dev="cuda"):
    c, st = case, prepare(case, seed, dev)
    if c["op"] == "rotary":
        turn = torch.polar(torch.full((1,), c["scale"], dtype=torch.float64, device=dev),
                           (-1 if c["inverse"] else 1) * torch.outer(st["pos"].double(), st["freq"].double()))[:, None]
        out, R = st["x"].double(), c["part"]
        i = torch.arange(R // 2, device=dev)
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
        z = torch.complex(out[..., a], out[..., b]) * turn
        out[..., a], out[..., b] = z.real, z.imag
        return out
    n, lengths = _ragged(c)
    table, ps = st["table"].tolist(), c["page"]
    if c["op"] == "append":
        out = []
        for x in (st["k"], st["v"]):
            parts = x.double().split(GROUP, -1)
            scales = [(p.abs().max(-1, keepdim=True).values / 7).to(torch.bfloat16).double() for p in parts]
            out.append(torch.cat([torch.nan_to_num(p / s).round().clamp(-7, 7) * s for p, s in zip(parts, scales)], -1))
        return tuple(out)
    at = lambda s, rows: (st["table"][s].long()[rows // ps], rows % ps)  # noqa: E731
    if c["op"] == "evict":
        K, keep, D = c["heads"], c["keep"], c["dim"]
        kept = torch.full((c["seqs"], K, keep), -1, dtype=torch.int32, device=dev)
        k, v = (torch.zeros(c["seqs"], keep, K, D, dtype=torch.float64, device=dev) for _ in "kv")
        weights = st["weights"].double()
        for s, m in enumerate(lengths):
            rows = torch.arange(m, device=dev)
            page, place = at(s, rows)
            w, new = st["weights"][page, :, place].t().double(), min(m, keep)
            w[:, : _first(c)] = math.inf
            w[:, max(0, m - _recent(c)):] = math.inf
            order = torch.argsort(-w, dim=1, stable=True)[:, :new].sort(1).values
            kept[s, :, :new] = order.int()
            kv = [_row_values(st[x + "_codes"], st[x + "_scales"], page, place) for x in "kv"]
            into, ip = st["into"][s].long()[rows[:new] // ps], rows[:new] % ps
            for h in range(K):
                k[s, keep - new:, h], v[s, keep - new:, h] = kv[0][order[h], h], kv[1][order[h], h]
                weights[into, h, ip] = st["weights"][page, h, place].double()[order[h]]
        return kept, None, k.flatten(0, 1), v.flatten(0, 1), weights
    G, D, out = c["q_heads"] // c["heads"], c["dim"], []
    sums = st["weights"].double() if c["weights"] else None
    for s, m in enumerate(lengths):
        page, place = at(s, torch.arange(m, device=dev))
        k = _row_values(st["k_codes"], st["k_scales"], page, place)
        v = _row_values(st["v_codes"], st["v_scales"], page, place)
        first = sum(n[:s])
        q = st["q"][first: first + n[s]].double()
        here = torch.arange(m - n[s], m, device=dev)[:, None]
        key = torch.arange(m, device=dev)
        hidden = (key > here) | (key <= here - (c["window"] or m))
        o = torch.empty_like(q)
        for h in range(c["q_heads"]):
            z = (q[:, h] @ k[:, h // G].t() / math.sqrt(D)).masked_fill(hidden, -math.inf)
            p = torch.softmax(z, 1)
            o[:, h] = p @ v[:, h // G]
            if sums is not None:
                sums[page, h // G, place] += p.sum(0)
        out.append(o)
    return torch.cat(out) if sums is None else (torch.cat(out), sums)
