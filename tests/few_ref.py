"""The few-token products in fp64, with the error bounds their GPU tests use.

Bounds.  A sum of n fp32 terms accumulated in any order is off by at most
n u sum|terms| (u = 2^-24, one rounding per addition; 2u where the matrix cores'
own additions may cut off instead; products of a 16-bit float and a small
integer are exact in fp32).  The kernels sum at most 128 columns before the
scale multiplies the sum: 4 matrix instructions of 33 additions per plane of x,
and as many again for bf16 activations with 2-4 bits, which sum (2^b + q) x and
-(2^b + z) x as separate terms, larger than (q - z) x.  The scaled sums, one per
32 columns or more, are then added, and the sums of eight waves.  The result is
rounded once to its type: half an ulp, or half the smallest subnormal.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
EPS_HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}  # half a step, relative to the value
TINY_HALF = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def make_packed(rng, oracle, d_out, d_in, bits, group, perm=False, n=None):
    """A random packed layer (n: a stack): dict of host arrays."""
    lead = () if n is None else (n,)
    g = group or d_in
    codes = rng.integers(0, 2 ** bits, size=lead + (d_out, d_in), dtype=np.uint8)
    scales = rng.uniform(0.2, 1.0, size=lead + (d_out, d_in // g)).astype(np.float32) * np.float32(2.0 / (2 ** bits * np.sqrt(d_in)))
    zeros = rng.integers(0, 2 ** bits, size=lead + (d_out, d_in // g)).astype(np.float32)
    kperm = None
    if perm:
        kperm = np.stack([rng.permutation(d_in) for _ in range(n or 1)]).astype(np.int32)
        kperm = kperm if n is not None else kperm[0]
    flat = codes.reshape(-1, d_in)
    packed = oracle.pack_codes(flat, bits).reshape(lead + (d_out, -1))
    return dict(q=codes, packed=packed, scales=scales, zeros=zeros, kperm=kperm, bits=bits, group=group)


def matrix(w, e=None):
    """(W_hat, the magnitude of the summed terms per weight) in packed column order, fp64."""
    q, s, z = (w[k] if e is None else w[k][e] for k in ("q", "scales", "zeros"))
    gi = np.arange(q.shape[1]) // (w["group"] or q.shape[1])
    q, s, z = q.astype(np.float64), s.astype(np.float64)[:, gi], z.astype(np.float64)[:, gi]
    return (q - z) * s, (2.0 ** w["bits"] * 2 + q + z) * s


def product(x, w, e=None, dx=None, planes=1):
    """x [M][d_in] fp64 times the packed layer: (value, error bound of the fp32 sums), with an error dx of x and x
    given as a sum of `planes` terms."""
    order = w["kperm"] if e is None or w["kperm"] is None else w["kperm"][e]
    if order is not None:
        x = x[:, order]
        dx = None if dx is None else dx[:, order]
    W, A = matrix(w, e)
    per_fold = 2 * 2 * planes * min(4, x.shape[1] // 32) * 33 * U * 1.01  # (the planes of x add up to a little more than |x|)
    folds = (x.shape[1] // 32 + 16) * U
    bound = np.abs(x) @ (per_fold * A + folds * np.abs(W)).T
    if dx is not None:
        bound = bound + dx @ (np.abs(W) * (1 + folds) + per_fold * A).T
    return x @ W.T, bound


def rounded(v, bound, out):
    """The bound after the result's rounding to `out`."""
    return bound + EPS_HALF[out] * (np.abs(v) + bound) + TINY_HALF[out]


def silu_mul(g, dg, u, du):
    """silu(g) u and its bound: |silu'| <= 1.1; exp, the division and two products within 8 ulp of fp32."""
    with np.errstate(over="ignore"):
        sg = g / (1.0 + np.exp(-g))
    v = sg * u
    dv = 1.1 * dg * np.abs(u) + np.abs(sg) * du + 1.1 * dg * du
    return v, dv + 16 * U * (np.abs(v) + dv)


def route(x, router, top_k, renormalize):
    """(ids, weights) of the router in fp64; descending logits, ties to the lower index."""
    logits = x @ router.T
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    w = np.take_along_axis(p, ids, axis=1)
    return ids.astype(np.int32), w / w.sum(axis=1, keepdims=True) if renormalize else w


def moe(x, gate, up, down, ids, weights, out):
    """The experts' sum for x [T][d] in fp64 with h rounded nowhere, and the bound that counts its pieces: two bf16
    terms (2^-8 of 2^-8 of it is lost) for a 16-bit result, three for fp32."""
    planes = 3 if out == "fp32" else 2
    T, k = ids.shape
    E = gate["q"].shape[0]
    y = np.zeros((T, down["q"].shape[1]))
    b = np.zeros_like(y)
    mag = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            g, dg = product(x[t:t + 1], gate, e)
            u, du = product(x[t:t + 1], up, e)
            h, dh = silu_mul(g, dg, u, du)
            dh = dh + 2.0 ** (-8 * planes) * (np.abs(h) + dh)
            v, dv = product(h, down, e, dh, planes)
            w = abs(float(weights[t, j]))
            y[t] += float(weights[t, j]) * v[0]
            b[t] += w * dv[0]
            mag[t] += w * (np.abs(v[0]) + dv[0])
    # the weight's own rounding and product, the waves' sums (a handful of additions per expert)
    return y, rounded(y, b + (16 + 4 * k) * U * mag, out)
