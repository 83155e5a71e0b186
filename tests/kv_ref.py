"""The 4-bit cache and the attention over it in 64 bits, row by row: what the
GPU tests of them compare with.  Everything here runs on the CPU."""
import numpy as np
import torch

U = 2.0 ** -24  # half a step of float32, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def quantise(x):
    """(codes [..., D], scales [..., D / 64] bf16) of x [..., D], in float64."""
    v = x.double().unflatten(-1, (-1, 64))
    s = (v.abs().amax(-1) / 7).float().bfloat16()
    q = torch.where(s.unsqueeze(-1) > 0, v / s.double().unsqueeze(-1), 0.0).round().clamp(-7, 7)
    bad = ~torch.isfinite(v).all(-1)
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    return torch.where(bad.unsqueeze(-1), torch.zeros_like(q), q).flatten(-2), s


def pack(q):
    q = q.to(torch.int64) & 15
    return (q[..., 0::2] | q[..., 1::2] << 4).to(torch.uint8)


def unpack(b):
    b = b.to(torch.int64)
    q = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return (q - 16 * (q > 7)).double()


class Pool:
    """A cache on the CPU whose places hold junk (NaN scales) until written,
    and tables whose unused entries name no page."""

    def __init__(self, lengths, heads, dim, page, seed=0, spare=0, capacity=None):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.dim, self.page, self.lengths = heads, dim, page, list(lengths)
        S, most = len(lengths), max(max(lengths), 1)
        width = -(-max(most, capacity or 0) // page)
        need = [-(-n // page) for n in lengths]
        more = -(-spare // page)
        self.pages = sum(need) + S * more + 2
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((S, width + 1), -1, dtype=torch.int32)
        self.table[:, width] = 1 << 30
        at = 0
        for s in range(S):
            self.table[s, : need[s]] = order[at: at + need[s]]
            at += need[s]
        self.into = order[at: at + S * more].view(S, more) if more else None
        shape = (self.pages, heads, page)
        junk = lambda: torch.randint(0, 256, (*shape, dim // 2), generator=g).to(torch.uint8)  # noqa: E731
        self.k_codes, self.v_codes = junk(), junk()
        self.k_scales = torch.full((self.pages, heads, dim // 64, page), float("nan"), dtype=torch.bfloat16)
        self.v_scales = self.k_scales.clone()
        self.weights = torch.rand(shape, generator=g)

    def place(self, s, row):
        """(page, slot) of a row, None where there is none."""
        i = row // self.page
        if row < 0 or i >= self.table.shape[1] or not 0 <= int(self.table[s, i]) < self.pages:
            return None
        return int(self.table[s, i]), row % self.page

    def write(self, s, row, k, v):
        p = self.place(s, row)
        if p is None:
            return
        for codes, scales, x in ((self.k_codes, self.k_scales, k), (self.v_codes, self.v_scales, v)):
            q, sc = quantise(x)
            codes[p[0], :, p[1]] = pack(q)
            scales[p[0], :, :, p[1]] = sc

    def fill(self, seed=1, v_gain=None):
        """Random keys and values in every row; v_gain(s, row) multiplies a row's values."""
        g = torch.Generator().manual_seed(seed)
        for s, n in enumerate(self.lengths):
            for r in range(n):
                k = torch.randn(self.heads, self.dim, generator=g) * torch.exp(0.5 * torch.randn(self.heads, 1, generator=g))
                v = torch.randn(self.heads, self.dim, generator=g) * torch.exp(0.5 * torch.randn(self.heads, 1, generator=g))
                self.write(s, r, k, v * (v_gain(s, r) if v_gain else 1.0))
        return self

    def rows(self, s, n):
        """(k, v float64 [n, heads, D], k and v scales [n, heads, D / 64], there [n]) of a sequence's first n rows."""
        out = [torch.zeros(n, self.heads, self.dim, dtype=torch.float64) for _ in "kv"]
        sc = [torch.zeros(n, self.heads, self.dim // 64, dtype=torch.float64) for _ in "kv"]
        there = torch.zeros(n, dtype=torch.bool)
        for r in range(n):
            p = self.place(s, r)
            if p is None:
                continue
            there[r] = True
            for i, (c, z) in enumerate(((self.k_codes, self.k_scales), (self.v_codes, self.v_scales))):
                sc[i][r] = z[p[0], :, :, p[1]].double()
                out[i][r] = unpack(c[p[0], :, p[1]]) * sc[i][r].repeat_interleave(64, -1)
        return out[0], out[1], sc[0], sc[1], there

    def to(self, dev, cm, weights=True):
        return cm.KVCache(self.k_codes.to(dev), self.k_scales.to(dev), self.v_codes.to(dev), self.v_scales.to(dev),
                          self.weights.to(dev) if weights else None)


def attention(pool, q, new, scale=None, window=0):
    """(out [T, Hq, D], tolerance, weights per place, their tolerance) of queries q [T, Hq, D], `new` of each sequence
    being its last rows.

    Tolerances, with U = 2^-24: a score is a float32 sum of D products of a query element and a code of at most 8, in
    steps of 32 that are added against their largest, so it is off by at most (D + 64) U 8 sum |q| s_k scale, and by
    8 U of itself and of the maximum it is taken off from; a weight is off by that times itself, twice with the
    normaliser's.  The weights go into the product with 11 bits (bf16) or 22 (f16), and the product's float32 sum over
    n keys (codes of at most 8, times weight times scale) is off by (n + 128) U of its size.  The result is rounded once
    (half precision: to 2^-25 at least)."""
    T, Hq, D = q.shape
    floor = 2.0 ** -25 if q.dtype == torch.float16 else 0.0
    G = Hq // pool.heads
    scale = D ** -0.5 if scale is None else scale
    out, tol = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    w, wtol = torch.zeros(pool.weights.shape, dtype=torch.float64), torch.zeros(pool.weights.shape, dtype=torch.float64)
    h = HALF_STEP[q.dtype]
    bits = 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -21
    t = 0
    for s, n in enumerate(new):
        length = pool.lengths[s]
        k, v, ks, vs, there = pool.rows(s, length)
        for i in range(n):
            pos = length - n + i
            seen = there.clone()
            key = torch.arange(length)
            seen &= key <= pos
            if window:
                seen &= key > pos - window
            at = torch.nonzero(seen)[:, 0]
            for hh in range(Hq):
                if len(at) == 0:
                    continue
                x, kh = q[t, hh].double(), hh // G
                z = (k[at, kh] @ x) * scale
                p = torch.softmax(z, 0)
                mass = (x.abs().view(-1, 64).sum(1) * ks[at, kh].abs()).sum(1) * abs(scale)
                zm = z.abs().max()
                d = float((U * ((D + 64) * 8 * mass + 8 * 1.5 * (z.abs() + zm))).max()) + 8 * U
                o = p @ v[at, kh]
                a = p @ v[at, kh].abs()
                b = (p @ vs[at, kh].abs()).repeat_interleave(64)
                out[t, hh] = o
                tol[t, hh] = h * o.abs() + floor + (bits + 2 * d) * a + (len(at) + 128) * U * 8 * b + 2.0 ** -36 * b
                for r, pr in zip(at.tolist(), p.tolist()):
                    pl = pool.place(s, r)
                    w[pl[0], kh, pl[1]] += pr
                    wtol[pl[0], kh, pl[1]] += (2 * d + (len(at) + 64) * U) * pr
            t += 1
    return out, tol, w, wtol + (T * G + 32) * U * w


def offsets_of(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
