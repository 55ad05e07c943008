"""What the errors of the few-token products may be on random data: a bound of their root mean square, beside the bounds
of the worst case in few_ref.py, which are two to four orders of magnitude wider.

The terms of a sum here have random signs (activations are symmetric about zero), so its partial sums are about the root
of the sum of squares, and its n roundings, each of at most u |partial sum| (2 u where the matrix cores may cut off),
add up as a random walk, not linearly.  With the counts of few_ref.py (264 additions per plane of x and 128 columns, one
of scaled sums per 32 columns and for eight waves): sigma^2 = 264 planes (2u)^2 sum (A x)^2 + folds u^2 sum (W x)^2,
where A is the magnitude of a weight's terms before they cancel.  Errors of different hidden values are independent, as
their weights are different rows.  The root mean square of error / sigma is at most 1."""
from __future__ import annotations

import numpy as np

import few_ref as fr


def product(x, w, e=None, var_x=None, planes=1):
    """(x W^T, the variance of its error): x [M][d_in] fp64 with errors of variance var_x."""
    order = w["kperm"] if e is None or w["kperm"] is None else w["kperm"][e]
    if order is not None:
        x = x[:, order]
        var_x = None if var_x is None else var_x[:, order]
    W, A = fr.matrix(w, e)
    folds = x.shape[1] // 32 + 16
    var = 264 * planes * (2 * fr.U) ** 2 * (x ** 2 @ (A ** 2).T) + folds * fr.U ** 2 * (x ** 2 @ (W ** 2).T)
    if var_x is not None:
        var = var + var_x @ (W ** 2).T
    return x @ W.T, var


def silu_mul(g, var_g, u, var_u):
    v, _ = fr.silu_mul(g, 0.0, u, 0.0)
    s = fr.silu_mul(g, 0.0, np.ones_like(u), 0.0)[0]
    return v, (1.1 * u) ** 2 * var_g + s ** 2 * var_u + (16 * fr.U * v) ** 2


def gated(x, gate, up, e=None):
    return silu_mul(*product(x, gate, e), *product(x, up, e))


def moe(x, gate, up, down, ids, weights, planes):
    """The experts' sum, h held in `planes` bf16 values between the products (2^-8 is left of each)."""
    y = np.zeros((x.shape[0], down["q"].shape[1]))
    var = np.zeros_like(y)
    for e in np.unique(ids):
        if not 0 <= e < gate["q"].shape[0]:
            continue
        t, j = np.nonzero(ids == e)
        h, var_h = gated(x[t], gate, up, e)
        v, var_v = product(h, down, e, var_h + (2.0 ** (-8 * planes) * h) ** 2, planes)
        w = weights[t, j][:, None]
        np.add.at(y, t, w * v)
        np.add.at(var, t, w ** 2 * var_v + ((16 + 4 * ids.shape[1]) * fr.U * w * v) ** 2)
    return y, var


def rms(got, want, var, out="fp32"):
    """The root mean square of error / sigma, with the result's rounding to `out`."""
    var = var + (fr.EPS_HALF[out] * want) ** 2 + fr.TINY_HALF[out] ** 2
    return float(np.sqrt(np.mean((got - want) ** 2 / var)))
