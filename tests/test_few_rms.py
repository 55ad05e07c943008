"""The bounds of few_rms.py are passed by results rounded to fp32 and show mistakes planted in the formulas."""
import numpy as np
import pytest

import few_ref as fr
import few_rms


def _bf16(v):
    m, e = np.frexp(v)
    return np.ldexp(np.round(m * 256), e - 8)


@pytest.mark.parametrize("bits,group,d,ff", [(4, 32, 256, 160), (4, 128, 512, 1024), (8, 0, 416, 256), (2, 64, 512, 384), (3, 32, 4096, 96)])
def test_planted_mistakes_show(oracle_mod, bits, group, d, ff):
    rng = np.random.default_rng(bits + d)
    E, T, k = 4, 6, 2
    gate, up = (fr.make_packed(rng, oracle_mod, ff, d, bits, group, n=E) for _ in range(2))
    down = fr.make_packed(rng, oracle_mod, d, ff, bits, group, n=E)
    x = _bf16(rng.standard_normal((T, d)))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = rng.uniform(0.1, 1, size=ids.shape)
    want, var = few_rms.moe(x, gate, up, down, ids, weights, 3)

    def layer(gate=gate, up=up, down=down, piece=lambda h: h):
        y = np.zeros_like(want)
        for t in range(T):
            for j in range(k):
                h = piece(few_rms.gated(x[t:t + 1], gate, up, ids[t, j])[0])
                y[t] += weights[t, j] * few_rms.product(h, down, ids[t, j])[0][0]
        return y.astype(np.float32)

    def scales(w):
        return dict(w, scales=_bf16(w["scales"].astype(np.float64)).astype(np.float32))

    def without_last(w):
        q = w["q"].copy()
        q[..., -1] = w["zeros"][..., -1].astype(np.uint8)
        return dict(w, q=q)

    assert few_rms.rms(layer(), want, var) < 0.1
    for mistake in (dict(piece=_bf16), dict(gate=scales(gate)), dict(up=scales(up)), dict(down=scales(down)),
                    dict(gate=without_last(gate)), dict(up=without_last(up)), dict(down=without_last(down))):
        assert few_rms.rms(layer(**mistake), want, var) > 10
