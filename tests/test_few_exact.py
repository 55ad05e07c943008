"""The exact layers of few_exact.py show mistakes: planted in the formulas, each changes a result."""
import numpy as np
import pytest

import few_exact as fx
import few_ref as fr


def _hidden(x, gate, up, e):
    return fr.product(x, gate, e)[0] * fr.product(x, up, e)[0]


def _without(w, col):
    """The layer without a packed column."""
    q = w["q"].copy()
    q[..., col] = np.repeat(w["zeros"], w["group"] or q.shape[-1], axis=-1)[..., col].astype(np.uint8)
    return dict(w, q=q)


@pytest.mark.parametrize("bits,group,perm", [(2, 32, True), (3, 32, False), (4, 64, True), (8, 0, False), (4, 128, False)])
def test_planted_mistakes_show(oracle_mod, bits, group, perm):
    rng = np.random.default_rng(bits)
    T, d, ff = 16, 256, 640
    gate, up, down = fx.experts(rng, oracle_mod, 1, d, ff, bits, group, perm, True)
    x = fx.acts(rng, T, d)
    want, n_pieces = fx.moe(x, gate, up, down, np.zeros((T, 1), dtype=np.int32), np.ones((T, 1)))
    h = _hidden(x, gate, up, 0)
    assert n_pieces == 3
    out = lambda h, w=down: fr.product(h, w, 0)[0].astype(np.float32)  # noqa: E731
    assert np.array_equal(out(h), want)
    for n in (1, 2):
        assert not np.array_equal(out(fx.pieces(h, n)), want)
    for col in (0, ff - 1):
        assert (out(h, _without(down, col)) != want).any(axis=1).all()
    for col in (0, d - 1):
        assert not np.array_equal(out(_hidden(x, _without(gate, col), up, 0)), want)
        assert not np.array_equal(out(_hidden(x, gate, _without(up, col), 0)), want)
    late = dict(down, zeros=down["zeros"].copy())
    late["zeros"][0, :, -1] += 1
    assert not np.array_equal(out(h, late), want)


def test_integers_of_16_bits_for_16_bit_results(oracle_mod):
    rng = np.random.default_rng(1)
    gate, up, down = fx.experts(rng, oracle_mod, 2, 128, 640, 4, 32, False, False)
    x = fx.acts(rng, 6, 128)
    _, n_pieces = fx.moe(x, gate, up, down, rng.integers(0, 2, size=(6, 1)), np.ones((6, 1)))
    assert n_pieces == 2


@pytest.mark.parametrize("out", ["bf16", "fp16"])
def test_pieces_of_h_show_in_16_bit_results(oracle_mod, out):
    """Two bf16 values for h change roundings of the cases with 16-bit results; three do not."""
    torch = pytest.importorskip("torch")
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[out]
    rng = np.random.default_rng(16 + 4096 + 640 + 3)
    gate, up, down = fx.experts(rng, oracle_mod, 2, 4096, 640, 3, 32, False, True)
    if out == "fp16":
        down["scales"] = down["scales"] / np.float32(512)
    x = fx.acts(rng, 16, 4096)
    h = _hidden(x, gate, up, 0)
    y = [torch.from_numpy(fr.product(fx.pieces(h, n), down, 0)[0].astype(np.float32)).to(dt) for n in (2, 3)]
    want = torch.from_numpy(fr.product(h, down, 0)[0].astype(np.float32)).to(dt)
    assert not torch.equal(y[0], want) and torch.equal(y[1], want)
