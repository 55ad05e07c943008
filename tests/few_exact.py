"""Layers of small integers on which gemv_gated and moe_layer are exact: every sum of magnitudes stays below 2^24 units, so
fp32 holds every partial sum in any order, every gate is at least 32, where fp32 has silu(g) = g (1 + exp(-32) rounds to
1), and scales are powers of two.  What is left is the result's rounding, so a kernel is compared to the bit: a
column, a code, a zero, a scale or a piece of h that is lost or counted twice shows."""
from __future__ import annotations

import numpy as np

import few_ref as fr

UNITS = 2.0 ** 24


def _layer(rng, oracle, shape, bits, group, perm, low, high, count, scales, z_top):
    """Codes z + c with c from max(low, -z) to min(high, top - z) at `count` columns of a row, and z elsewhere."""
    top = 2 ** bits - 1
    *lead, d_out, d_in = shape
    g = group or d_in
    z = rng.integers(0, z_top + 1, size=(*lead, d_out, d_in // g))
    zc = np.repeat(z, g, axis=-1)
    low, high = np.maximum(low, -zc), np.minimum(high, top - zc)
    c = np.where(low <= high, rng.integers(np.minimum(low, high), high + 1), 0)
    if count < d_in:
        r = rng.random(c.shape, dtype=np.float32)
        r[..., [0, -1]] = 0  # the first and the last packed column are among them
        c = np.where(r <= np.partition(r, count - 1, axis=-1)[..., count - 1:count], c, 0)
    s = rng.choice(np.array(scales, dtype=np.float32), size=z.shape)
    kperm = None
    if perm:
        n = int(np.prod(lead)) if lead else 1
        kperm = np.stack([rng.permutation(d_in) for _ in range(n)]).astype(np.int32).reshape(*lead, d_in)
    w = dict(c=c, q=(zc + c).astype(np.uint8), scales=s, zeros=z.astype(np.float32), kperm=kperm, bits=bits, group=group)
    return pack(w, oracle)


def pack(w, oracle):
    w["packed"] = oracle.pack_codes(np.ascontiguousarray(w["q"].reshape(-1, w["q"].shape[-1])), w["bits"]).reshape(*w["q"].shape[:-1], -1)
    return w


def gate_and_up(rng, oracle, shape, bits, group, perm, large):
    """A gate whose results are some hundreds, and an up matrix whose results are of both signs: their products have up
    to 19 bits (large) or 15."""
    gate = _layer(rng, oracle, shape, bits, group, perm, 1, 2, 32 if large else 24, (1, 2) if large else (1,), 2 ** bits - 2)
    # the codes of a row are all above or all below their zero: most hidden values are then nearly as large as the largest
    above = rng.random((*shape[:-1], 1)) < 0.5
    count = {2: 120, 3: 56, 4: 27, 8: 44}[bits] if large else 3
    up = _layer(rng, oracle, shape, bits, group, perm, np.where(above, 1, -7), np.where(above, 7, -1), count,
                (1, 2) if large else (1,), 2 ** bits - 1)
    up["kperm"] = gate["kperm"]
    return gate, up


def acts(rng, M, d_in):
    return rng.integers(1, 8, size=(M, d_in)).astype(np.float64)


def _summed(w, x, e=None):
    """The largest value that any order of a product's additions may reach, in units of its terms: in a step as the matrix
    cores see it (a column adds (q - z) x, or with 2-4 bits of bf16 (2^b + q) x and -(2^b + z) x, one after the other),
    and over the whole scaled row."""
    W = fr.matrix(w, e)[0]
    z = np.repeat(w["zeros"] if e is None else w["zeros"][e], w["group"] or W.shape[1], axis=-1)
    q = w["q"] if e is None else w["q"][e]
    A = np.abs(q - z) if w["bits"] == 8 else 2.0 ** w["bits"] + np.maximum(q, z)
    order = w["kperm"] if e is None or w["kperm"] is None else w["kperm"][e]
    xp = np.abs(x if order is None else x[:, order])
    s = w["scales"] if e is None else w["scales"][e]
    steps = [(xp[:, k:k + 128] @ A[:, k:k + 128].T).max() for k in range(0, xp.shape[1], 128)]
    return max(max(steps), (xp @ np.abs(W).T).max() / s.min())


def gated(x, gate, up, e=None):
    """silu(G) U, exact."""
    assert max(_summed(gate, x, e), _summed(up, x, e)) < UNITS
    G, U = fr.product(x, gate, e)[0], fr.product(x, up, e)[0]
    assert G.min() >= 32 and np.abs(G * U).max() < UNITS
    return G * U


def pieces(h, n):
    """The sum of n bf16 values next to h, each what the ones before leave."""
    got = np.zeros_like(h)
    for _ in range(n):
        m, e = np.frexp(h - got)
        got = got + np.ldexp(np.round(m * 256), e - 8)  # 8 significant bits
    return got


def experts(rng, oracle, E, d, ff, bits, group, perm, large):
    """Stacks whose hidden values are zero but at up to six packed columns of the second product, the first and the last
    among them, each in another step of 128 (one of them where there is one step); there the second product's codes are
    z + 1 or z - 1."""
    gate, up = gate_and_up(rng, oracle, (E, ff, d), bits, group, perm, large)
    top = 2 ** bits - 1
    down = _layer(rng, oracle, (E, d, ff), bits, group, perm, -top, top, ff, (1, 2), top)
    for e in range(E):
        steps = (ff + 127) // 128
        inner = rng.permutation(np.arange(1, steps - 1))[:4] if steps > 2 else np.array([], dtype=int)
        ends = [0, ff - 1] if steps > 1 else [rng.choice([0, ff - 1])]
        at = np.unique(np.concatenate([ends, 128 * inner + rng.integers(0, 128, size=len(inner))]).astype(int))
        live = at if down["kperm"] is None else down["kperm"][e][at]
        mask = np.zeros(ff, dtype=bool)
        mask[live] = True
        up["q"][e][~mask] = np.repeat(up["zeros"][e], (group or d), axis=-1)[~mask].astype(np.uint8)
        z = np.repeat(down["zeros"][e], (group or ff), axis=-1)[:, at]
        one = np.where(z == 0, 1, np.where(z == top, -1, rng.choice([-1, 1], size=z.shape)))
        down["q"][e][:, at] = (z + one).astype(np.uint8)
    return gate, pack(up, oracle), pack(down, oracle)


def moe(x, gate, up, down, ids, weights):
    """(the experts' sum, the bf16 values that every hidden value is a sum of: 1 to 3), exact."""
    E = gate["q"].shape[0]
    y = np.zeros((x.shape[0], x.shape[1]))
    mag, most = np.zeros_like(y), 1
    for e in range(E):
        rows = np.unique(np.nonzero(ids == e)[0])
        if len(rows) == 0:
            continue
        h = gated(x[rows], gate, up, e)
        most = next(n for n in range(most, 4) if np.array_equal(pieces(h, n), h))
        assert _summed(down, h, e) < UNITS / 1.02  # (the pieces of h add up to a little more than |h|)
        v = fr.product(h, down, e)[0]
        w = (np.where(ids[rows] == e, weights[rows], 0)).sum(axis=1, keepdims=True)
        y[rows] += w * v
        mag[rows] += np.abs(w * v)
    assert mag.max() < UNITS
    return y, most
