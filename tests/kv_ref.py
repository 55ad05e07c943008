"""The 4-bit key/value cache in numpy: its layout, its grids and, in 64 bits, what attention over it is, with bounds for the
kernels' errors.  Shares no code with the library."""
from __future__ import annotations

import numpy as np

HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}  # a rounding, relative
TERM = {"fp16": 2.0 ** -21, "bf16": 2.0 ** -11}  # of p s_v, by the result: two fp16 values (each to half a step) or one


def bf16_round(x: np.ndarray) -> np.ndarray:
    """fp32 rounded to bf16, ties to even (finite values and infinities)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def fit(x: np.ndarray, group: int, symmetric: bool):
    """Codes (u8, x's shape), scales and zeros ([..., groups]) of the last axis, in binary32."""
    f = np.float32
    x = x.astype(f)
    g = x.reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        if symmetric:
            s = np.abs(g).max(-1, keepdims=True) * (f(1) / f(7))
        else:
            lo, hi = np.minimum(g.min(-1, keepdims=True), f(0)), np.maximum(g.max(-1, keepdims=True), f(0))
            s = (hi - lo) * (f(1) / f(15))
        bad = ~np.isfinite(g).all(-1, keepdims=True)
        s = bf16_round(np.where(np.isfinite(s), s, f(np.inf)))
        s = np.where(s == 0, f(1), s)
        bad |= ~np.isfinite(s)
        if symmetric:
            z = np.full_like(s, 8)
            q = np.clip(np.rint(g / s), -7, 7) + f(8)
        else:
            z = np.clip(np.rint(-lo / s), 0, 15).astype(f)
            q = np.clip(np.rint(g / s + z), 0, 15)
        z = np.where(bad, f(8), z)
        q = np.where(bad, f(8), q)
        s = np.where(bad, f(np.nan), s)
    return q.astype(np.uint8).reshape(x.shape), s[..., 0].astype(f), z[..., 0].astype(f)


def grid_words(s: np.ndarray, z: np.ndarray) -> np.ndarray:
    hi = np.where(np.isnan(s), np.uint32(0x7FC0), np.ascontiguousarray(s).view(np.uint32) >> 16)
    lo = (8 - z).astype(np.float16).view(np.uint16).astype(np.uint32)
    return ((hi << 16) | lo).astype(np.uint32).view(np.int32)


def key_words(q: np.ndarray) -> np.ndarray:
    """Codes [..., D] -> int32 [..., D/8]."""
    D = q.shape[-1]
    w = np.zeros(q.shape[:-1] + (D // 8,), dtype=np.uint32)
    for d in range(D):
        t, b, e = d // 32, d // 8 % 4, d % 8
        w[..., b * (D // 32) + t] |= q[..., d].astype(np.uint32) << np.uint32(4 * (e // 2 + 4 * (e % 2)))
    return w.view(np.int32)


def value_units(q: np.ndarray) -> np.ndarray:
    """Codes [..., P, D] -> int16 [..., P/8, D/4, 8]."""
    *lead, P, D = q.shape
    v = np.zeros((*lead, P // 8, D // 4, 8), dtype=np.uint16)
    for d in range(D):
        u, j, m = d // 64, d // 16 % 4, d % 16
        v[..., 16 * u + m, :] |= (q[..., d].reshape(*lead, P // 8, 8).astype(np.uint16) << np.uint16(4 * j))
    return v.view(np.int16)


class Pool:
    """A pool in parts: codes [pages][H][P][D], scales and zeros [pages][H][P][groups], weight [pages][H][P]."""

    def __init__(self, pages, heads, dim, page, group, symmetric, seed=0, weights=True):
        rng = np.random.default_rng(seed)
        self.group, self.symmetric, self.dim, self.page, self.heads = group or dim, symmetric, dim, page, heads
        shape = (pages, heads, page, dim)
        ng = dim // self.group
        self.kq, self.vq = (rng.integers(0, 16, shape).astype(np.uint8) for _ in range(2))
        self.ks, self.vs = (bf16_round(np.exp(rng.normal(-2.5, 0.5, shape[:3] + (ng,))).astype(np.float32)) for _ in range(2))
        self.kz, self.vz = ((np.full(shape[:3] + (ng,), 8) if symmetric else rng.integers(5, 11, shape[:3] + (ng,))).astype(np.float32)
                            for _ in range(2))
        self.weight = rng.exponential(2.0, shape[:3]).astype(np.float32) if weights else None

    def words(self):
        """The five tensors, as numpy arrays."""
        grids = [grid_words(s, z).transpose(0, 1, 3, 2).copy() for s, z in ((self.ks, self.kz), (self.vs, self.vz))]
        return [key_words(self.kq), value_units(self.vq), *grids, None if self.weight is None else self.weight.copy()]

    def seq(self, row, n, name):
        """(codes, scales, zeros) of a table row's first n tokens: [H][n][...]; tokens on no page of the pool: there False."""
        slot = np.arange(n)
        page, at = np.asarray(row)[slot // self.page], slot % self.page
        there = (page >= 0) & (page < self.kq.shape[0])
        page = np.where(there, page, 0)
        q, s, z = (getattr(self, name + c)[page, :, at] for c in "qsz")  # [n][H][..]
        return q.transpose(1, 0, 2), s.transpose(1, 0, 2), z.transpose(1, 0, 2), there


def cuda_cache(gq, torch, pool):
    w = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in pool.words()]
    return gq.kv_cache(*w, group_size=pool.group, symmetric=pool.symmetric)


def attention(pool, q, table, lens, scale, dt, decay=None):
    """q [B][n][Hq][D] (values that fp16 or bf16 hold) in 64 bits: o, a bound of its error without the result's own rounding
    (TERM of every p s_v, and the fp32 sums'), the root-mean-square size of what TERM
    leaves, the weights [pages][H][P] and their bound."""
    B, n, Hq, D = q.shape
    H, G, g = pool.heads, Hq // pool.heads, pool.group
    o, tol, rms = (np.zeros(q.shape) for _ in range(3))
    weight = None if pool.weight is None else pool.weight.astype(np.float64)
    wtol = None if weight is None else np.zeros_like(weight)
    e24 = 2.0 ** -24
    for b in range(B):
        m = min(max(int(lens[b]), 0), len(table[b]) * pool.page)
        if m == 0:
            continue
        kq, ks, kz, there = pool.seq(table[b], m, "k")
        vq, vs, vz, _ = pool.seq(table[b], m, "v")
        ks, kz, vs, vz = (np.repeat(t.astype(np.float64), g, axis=2) for t in (ks, kz, vs, vz))
        k, v = ks * (kq - kz), vs * (vq - vz)
        # what the sums run over: q x and z x, q p s and z p s
        kmag, vmag = ks * (kq + kz), vs * (vq + vz)
        got, gtol = np.zeros((H, m)), np.zeros((H, m))
        for i in range(n):
            see = (np.arange(m) < m - n + 1 + i) & there
            if not see.any():
                continue
            x = q[b, i].reshape(H, G, D)
            s = scale * np.matmul(x, k.transpose(0, 2, 1))
            mag = scale * np.matmul(np.abs(x), kmag.transpose(0, 2, 1))
            s = np.where(see, s, -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            total = p.sum(-1, keepdims=True)
            p /= total
            # a score: D + 16 roundings of its magnitude; exp2 and its argument: 2^-21; sums over the tokens
            eps = (2 * ((D + 16) * e24 * np.where(see, mag, 0).max(-1, keepdims=True) + 2.0 ** -21) + m * e24)
            o[b, i] = np.matmul(p, v).reshape(Hq, D)
            small = 30 * np.where(see[:, None], vs, 0).max() * m * 2.0 ** -31 / total  # below fp16's normal numbers
            tol[b, i] = (np.matmul(p, np.abs(v)) * TERM[dt] + np.matmul(p, vmag) * eps + small).reshape(Hq, D)
            rms[b, i] = (TERM[dt] * np.sqrt(np.matmul(p * p, v * v)) + np.matmul(p, vmag) * eps + small).reshape(Hq, D)
            got += p.sum(1)
            gtol += (p * (eps + 2.0 ** -22)).sum(1)
        if decay is not None:
            slot = np.arange(m)[there]
            page, at = np.asarray(table[b])[slot // pool.page], slot % pool.page
            old = weight[page, :, at] if decay else 0.0
            weight[page, :, at] = decay * old + got[:, there].T
            wtol[page, :, at] = gtol[:, there].T + (n * G // 16 + 3) * e24 * np.abs(weight[page, :, at])
    return o, tol, rms, weight, wtol


def evict(pool, table, lens, to, budget, recent):
    """kept [B][H][budget], new lengths, and the pool's parts afterwards (a dict of copies)."""
    B, H, P = len(lens), pool.heads, pool.page
    parts = {k: getattr(pool, k).copy() for k in ("kq", "ks", "kz", "vq", "vs", "vz", "weight")}
    kept = np.full((B, H, budget), -1, dtype=np.int32)
    left = np.zeros(B, dtype=np.int32)
    pages = pool.kq.shape[0]
    for b in range(B):
        m = min(max(int(lens[b]), 0), len(table[b]) * P)
        keep = min(m, budget)
        late = min(recent, keep)
        left[b] = keep
        for h in range(H):
            def rank(i):
                page = table[b][i // P]
                w = float(pool.weight[page, h, i % P]) if 0 <= page < pages else float("nan")
                return (w == w, w if w == w else 0.0)
            order = sorted(range(m - late), key=lambda i: (tuple(-x for x in rank(i)), i))
            mine = sorted(order[:keep - late]) + list(range(m - late, m))
            kept[b, h, :keep] = mine
            for j, i in enumerate(mine):
                src, dst = table[b][i // P], to[b][j // P]
                if 0 <= src < pages and 0 <= dst < pages:
                    for a in parts:
                        parts[a][dst, h, j % P] = getattr(pool, a)[src, h, i % P]
    return kept, left, parts
