"""What is measured of the operators around the routed layer: the residual
addition with the root-mean-square norm, the dense product with its epilogue,
and the router's balance loss with its gradient.

A case names an operator ("op") and its sizes and types; prepare() makes its
inputs from a seed, run() is one pass (plain torch operations, or this
package's kernels where `own` is true), work() the bytes and operations that
a pass cannot do without, exact() the result in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
ALPHA = 1e-3
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "int8": torch.int8,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "int8": 1, "e4m3": 1}
QMAX = {"int8": 127.0, "e4m3": 448.0}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    norm, lin, bal = {"op": "norm"}, {"op": "linear"}, {"op": "balance"}
    return [
        # the layer's input while one token is decoded: latency alone
        dict(norm, name="norm one token", rows=1, hidden=6144, x="f32", residual="f32", out="f32", group=0),
        # a decode batch whose norm feeds an 8-bit product
        dict(norm, name="norm 64 rows int8", rows=64, hidden=6144, x="bf16", residual="f32", out="int8", group=0),
        # a ragged prompt in e4m3 with a scale per 128 columns, an odd row length (no 16-byte rows)
        dict(norm, name="norm ragged e4m3", rows=1531, hidden=2047, x="f16", residual="f16", out="e4m3", group=128),
        # a prefill batch, 16 bits in and out
        dict(norm, name="norm prefill", rows=4096, hidden=6144, x="bf16", residual="bf16", out="bf16", group=0),
        # one token through an 8-bit gate/up product with SwiGLU: the weights' bytes alone
        dict(lin, name="linear one token int8", m=1, n=2048, k=6144, type="int8", act="swiglu", bias=False,
             residual=False, out="bf16"),
        # a small decode batch, projection back to the hidden size onto the residual stream
        dict(lin, name="linear 16 rows", m=16, n=6144, k=2048, type="bf16", act="none", bias=True, residual=True,
             out="f32"),
        # a short ragged prompt, no size a multiple of a tile
        dict(lin, name="linear ragged", m=257, n=1001, k=2072, type="f16", act="gelu", bias=True, residual=False,
             out="f16"),
        # prefill products: 8-bit gate/up with SwiGLU, e4m3, and the 16-bit projection onto the residual
        dict(lin, name="linear prefill int8", m=4096, n=2048, k=6144, type="int8", act="swiglu", bias=False,
             residual=False, out="bf16"),
        dict(lin, name="linear prefill e4m3", m=4096, n=6144, k=2048, type="e4m3", act="none", bias=False,
             residual=True, out="bf16"),
        dict(lin, name="linear prefill bf16", m=4096, n=6144, k=6144, type="bf16", act="silu", bias=True,
             residual=True, out="bf16"),
        # one small batch's router, softmax scores; a training batch of ragged sequences with masked tokens
        dict(bal, name="balance small", tokens=64, experts=64, top_k=8, seqs=1, scores="softmax", masked=False, pad=0),
        dict(bal, name="balance batch", tokens=16384, experts=256, top_k=8, seqs=8, scores="sigmoid", masked=True,
             pad=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "balance"])
    if op == "norm":
        hidden = _log(rng, 64, 16384)
        rows = min(_log(rng, 1, 8192), 4096 * 6144 // hidden)
        x = rng.choice(["f32", "bf16", "f16"])
        return {"op": op, "rows": rows, "hidden": hidden, "x": x,
                "residual": rng.choice(["none", "f32", x]), "out": rng.choice(["f32", "bf16", "f16", "int8", "e4m3"]),
                "group": rng.choice([0, 0, 64, 128])}
    if op == "linear":
        n, k = _log(rng, 64, 8192), 16 * _log(rng, 4, 512)
        m = min(_log(rng, 1, 8192), 4096 * 6144 * 6144 // (2 * n * k))
        kind = rng.choice(["bf16", "f16", "int8", "e4m3"])
        return {"op": op, "m": m, "n": n, "k": k, "type": kind,
                "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5, "out": rng.choice(["f32", "bf16", "f16"])}
    experts = _log(rng, 2, 512)
    tokens = min(_log(rng, 1, 65536), 16384 * 256 // experts)
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, max(1, min(experts // 2, 16))),
            "seqs": min(_log(rng, 1, 64), tokens), "scores": rng.choice(["sigmoid", "softmax"]),
            "masked": rng.random() < 0.5, "pad": rng.choice([0, 0, 7])}


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["hidden"]
        b = n * (SIZE[c["x"]] + SIZE[c["out"]]) + 4 * c["hidden"]
        if c["residual"] != "none":
            b += 2 * n * SIZE[c["residual"]]
        if c["out"] in QMAX:
            b += 4 * c["rows"] * (-(-c["hidden"] // c["group"]) if c["group"] else 1)
        return {"bytes": b, "flops": 8 * n}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        wn = 2 * n if c["act"] == "swiglu" else n
        b = (m + wn) * k * SIZE[c["type"]] + m * n * SIZE[c["out"]] * (2 if c["residual"] else 1)
        b += 4 * (m + wn) if c["type"] in QMAX else 0
        b += 4 * wn if c["bias"] else 0
        return {"bytes": b, "flops": 2 * m * wn * k}
    T, E = c["tokens"] + c["pad"], c["experts"]
    # both directions: the logits for each, the choices once, the gradient, counts and loss
    return {"bytes": 3 * T * E * 4 + T * c["top_k"] * 4 + c["seqs"] * (E * 4 + 4), "flops": 24 * T * E}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _codes(rows, cols, kind, sigma, g, dev):
    """Rows quantised with a scale each, as weights and activations in 8 bits are."""
    v = torch.randn(rows, cols, generator=g, device=dev) * sigma
    s = v.abs().amax(1) / QMAX[kind]
    q = v / s[:, None]
    return (q.round_().clamp_(-127, 127) if kind == "int8" else q.clamp_(-448, 448)).to(TYPES[kind]), s


def prepare(case, seed, dev="cuda"):
    c, g = case, _gen(seed, dev)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if c["op"] == "norm":
        R, h = c["rows"], c["hidden"]
        st = dict(case=c, x=rnd(R, h).to(TYPES[c["x"]]), weight=1 + 0.1 * rnd(h))
        if c["group"]:
            st["group_of"] = torch.arange(h, device=dev) // c["group"]
        if c["residual"] != "none":
            # a residual stream: rows of different sizes, some columns larger than the rest
            r = rnd(R, h) * torch.exp(rnd(R, 1))
            r[:, :: max(1, h // 5)] *= 8
            st["residual"] = r.to(TYPES[c["residual"]])
            st["sum"] = torch.empty_like(st["residual"])
        return st
    if c["op"] == "linear":
        m, n, k, kind = c["m"], c["n"], c["k"], c["type"]
        wn = 2 * n if c["act"] == "swiglu" else n
        st = dict(case=c)
        if kind in QMAX:
            st["x"], st["x_scale"] = _codes(m, k, kind, 1.0, g, dev)
            st["w"], st["w_scale"] = _codes(wn, k, kind, 0.02, g, dev)
        else:
            st["x"], st["w"] = rnd(m, k).to(TYPES[kind]), (0.02 * rnd(wn, k)).to(TYPES[kind])
        st["bias"] = 0.1 * rnd(wn) if c["bias"] else None
        st["residual"] = rnd(m, n).to(TYPES[c["out"]]) if c["residual"] else None
        return st
    T, E, k, S = c["tokens"], c["experts"], c["top_k"], c["seqs"]
    rows = T + c["pad"]
    # a router that prefers some experts; the choices are the largest scores
    z = rnd(rows, E) + rnd(E)
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    drop = torch.rand(rows, k, generator=g, device=dev) < 0.05
    drop[:, 0] = False
    idx[drop] = -1
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device=dev)).values
    offsets = torch.cat([torch.zeros(1, device=dev, dtype=torch.long), cuts, torch.full((1,), T, device=dev)])
    mask = (torch.rand(rows, generator=g, device=dev) < 0.9) if c["masked"] else None
    if mask is not None:
        z[~mask] = float("nan")  # what stands in masked rows is never looked at
    return dict(case=c, logits=z, idx=idx, offsets=offsets.to(torch.int32), mask=mask, dloss=rnd(S),
                dlogits=torch.zeros(rows, E, device=dev))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _values(codes, scales, st):
    """8-bit rows as the values they stand for (16 bits hold them well)."""
    if scales.shape[1] > 1:
        scales = scales.index_select(1, st["group_of"])
    if codes.dtype != torch.int8:
        codes = codes.to(torch.bfloat16)  # exact
    return torch.mul(codes, scales, out=torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device))


def _quantise(y, kind, group):
    """Plain form of the 8-bit output: codes and scales of rows y (64 bits, since codes sit next to borders)."""
    R, h = y.shape
    g = group or h
    n = -(-h // g)
    yp = torch.nn.functional.pad(y, (0, n * g - h)).view(R, n, g)
    s = (yp.abs().amax(2, keepdim=True) / QMAX[kind]).float().double()
    q = torch.where(s > 0, yp / s, torch.zeros_like(yp))
    q = q.round().clamp(-127, 127).to(torch.int8) if kind == "int8" else q.clamp(-448, 448).float().to(TYPES[kind])
    return q.view(R, n * g)[:, :h], s.view(R, n).float()


def _act(v, act):
    if act == "relu":
        return torch.clamp_min(v, 0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    return v


def _epilogue(acc, st, c):
    if st["bias"] is not None:
        acc = acc + st["bias"]
    if c["act"] == "swiglu":
        g, u = acc[:, : c["n"]], acc[:, c["n"]:]
        acc = g * torch.sigmoid(g) * u
    else:
        acc = _act(acc, c["act"])
    return acc if st["residual"] is None else acc + st["residual"].to(acc.dtype)


def _scores(z, kind):
    """p (each row's shares), the scores and their row sums; rows of nothing give zeros."""
    if kind == "softmax":
        e = torch.exp(z - torch.nan_to_num(z.amax(1, keepdim=True), neginf=0.0))
    else:
        e = torch.sigmoid(z)
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e)), e, total


def _balance(st, c, dtype):
    """(loss, counts, dlogits) from the formulas, sums by products with 0/1 matrices."""
    T, E, S = st["logits"].shape[0], c["experts"], c["seqs"]
    rows = torch.arange(T, device=st["logits"].device)
    off = st["offsets"].long()
    member = (rows[None] >= off[:-1, None]) & (rows[None] < off[1:, None])
    if st["mask"] is not None:
        member = member & st["mask"][None]
    valid = member.any(0)
    member = member.to(dtype)
    z = torch.where(valid[:, None], st["logits"].to(dtype), torch.zeros((), dtype=dtype, device=off.device))
    p, e, total = _scores(z, c["scores"])
    seq = torch.where(valid, torch.searchsorted(off[1:].contiguous(), rows, right=True), 0)
    keep = (st["idx"] >= 0) & valid[:, None]
    slot = torch.where(keep, seq[:, None] * E + st["idx"], S * E)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=off.device)
    counts.index_add_(0, slot.reshape(-1), torch.ones_like(slot, dtype=torch.int32).reshape(-1))
    counts = counts[: S * E].view(S, E)
    n = counts.sum(1, keepdim=True).to(dtype)
    tokens = member.sum(1, keepdim=True)
    some = (n > 0) & (tokens > 0)
    coef = torch.where(some, ALPHA * E * counts.to(dtype) / (n.clamp_min(1) * tokens.clamp_min(1)), torch.zeros_like(n))
    loss = (coef * (member @ p)).sum(1)
    ct = coef[seq]
    d = ct - (ct * p).sum(1, keepdim=True)
    if c["scores"] == "softmax":
        d = p * d
    else:
        d = torch.where(total > 0, d * e * (1 - e) / total, torch.zeros_like(d))
    d = d * st["dloss"].to(dtype)[seq][:, None] * valid[:, None]
    return loss, counts, d


def run(state):
    st, c = state, state["case"]
    if own:
        import routed_expert_ffn_f32_amd as cm
        if c["op"] == "norm":
            got = cm.rms_norm(st["x"], st["weight"], EPS, residual=st.get("residual"), residual_out=st.get("sum"),
                              out_dtype=TYPES[c["out"]], group=c["group"])
            y = _values(got[0], got[1], st) if c["out"] in QMAX else got
            return (y, st["sum"]) if "sum" in st else (y,)
        if c["op"] == "linear":
            return cm.linear(st["x"], st["w"], x_scale=st.get("x_scale"), w_scale=st.get("w_scale"), bias=st["bias"],
                             act=c["act"], residual=st["residual"], out_dtype=TYPES[c["out"]])
        loss, counts, coef = cm.balance_loss(st["logits"], st["idx"], ALPHA, scores=c["scores"], offsets=st["offsets"],
                                             mask=st["mask"])
        d = cm.balance_grad(st["logits"], coef, st["dloss"], scores=c["scores"], offsets=st["offsets"],
                            mask=st["mask"], out=st["dlogits"])
        return loss, counts, d
    if c["op"] == "norm":
        s = st["x"].float()
        if "sum" in st:
            s = (s + st["residual"].float()).to(st["residual"].dtype)
            st["sum"].copy_(s)
        if c["out"] in QMAX:
            s = s.double()
            y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * st["weight"].double()
            y = _values(*_quantise(y, c["out"], c["group"]), st)
        else:
            s = s.float()
            y = (s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * st["weight"]).to(TYPES[c["out"]])
        return (y, st["sum"]) if "sum" in st else (y,)
    if c["op"] == "linear":
        acc = st["x"].float() @ st["w"].float().t()
        if "x_scale" in st:
            acc = acc * st["x_scale"][:, None] * st["w_scale"]
        return _epilogue(acc, st, c).to(TYPES[c["out"]])
    loss, counts, d = _balance(st, c, torch.float32)
    st["dlogits"].copy_(d)
    return loss, counts, st["dlogits"]


# ---------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def exact(case, seed, dev="cuda"):
    c, st = case, prepare(case, seed, dev)
    if c["op"] == "norm":
        v = st["x"].double()
        if "residual" in st:
            # the sum is kept in the residual's type, and that is what is normed
            v = (v + st["residual"].double()).to(st["residual"].dtype).double()
        y = st["weight"].double() * v / ((v * v).sum(1, keepdim=True) / c["hidden"] + EPS) ** 0.5
        if c["out"] in QMAX:
            parts = []
            for lo in range(0, c["hidden"], c["group"] or c["hidden"]):
                blk = y[:, lo:lo + (c["group"] or c["hidden"])]
                s = blk.abs().max(1, keepdim=True).values / QMAX[c["out"]]
                q = torch.nan_to_num(blk / s, nan=0.0)
                q = torch.round(q) if c["out"] == "int8" else q.float().to(torch.float8_e4m3fn).double()
                parts.append(q * s)
            y = torch.cat(parts, 1)
        return (y, v) if "residual" in st else (y,)
    if c["op"] == "linear":
        a = torch.matmul(st["x"].double(), st["w"].double().t())
        if "x_scale" in st:
            a = a * torch.outer(st["x_scale"].double(), st["w_scale"].double())
        if st["bias"] is not None:
            a = a + st["bias"].double()
        f = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v / (1 + torch.exp(-v)),
             "gelu": lambda v: v * (1 - torch.erfc(v / math.sqrt(2)) / 2),
             "gelu_tanh": lambda v: v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))}
        if c["act"] == "swiglu":
            a = f["silu"](a[:, : c["n"]]) * a[:, c["n"]:]
        else:
            a = f[c["act"]](a)
        return a if st["residual"] is None else a + st["residual"].double()
    # the balance loss, sequence by sequence
    E, off = c["experts"], st["offsets"].tolist()
    loss = torch.zeros(c["seqs"], dtype=torch.float64, device=dev)
    d = torch.zeros(st["logits"].shape, dtype=torch.float64, device=dev)
    for s in range(c["seqs"]):
        at = torch.arange(off[s], off[s + 1], device=dev)
        if st["mask"] is not None:
            at = at[st["mask"][at]]
        z, ids = st["logits"][at].double(), st["idx"][at]
        ids = ids[ids >= 0].long()
        if not len(at) or not len(ids):
            continue
        coef = ALPHA * E * torch.bincount(ids, minlength=E).double() / (len(ids) * len(at))
        if c["scores"] == "softmax":
            p = torch.softmax(z, 1)
            slope = p
        else:
            sg = 1 / (1 + torch.exp(-z))
            tot = sg.sum(1, keepdim=True)
            p, slope = sg / tot, sg * (1 - sg) / tot
        loss[s] = (p * coef).sum()
        d[at] = st["dloss"][s].double() * slope * (coef - (p @ coef)[:, None])
    return loss, None, d
