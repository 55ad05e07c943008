"""The 4-bit cache's layout and grids as the tests hold them (kv_ref.py): hand-made words, the grid's corner cases, and the
same bytes and values as the plain forms of perf/more_operators.py (which share no code with it)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plain():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_words_by_hand():
    q = np.zeros((1, 64), dtype=np.uint8)
    q[0, 0], q[0, 1], q[0, 7], q[0, 8], q[0, 32] = 1, 2, 3, 4, 5
    w = kv_ref.key_words(q).view(np.uint32)[0]
    # dim 0: bits 0; dim 1: bits 16; dim 7: bits 4 (3 + 4); dim 8: lane row 1, word 2; dim 32: step 1, word 1
    assert w.tolist() == [1 | 2 << 16 | 3 << 28, 5, 4, 0, 0, 0, 0, 0]
    v = np.zeros((8, 64), dtype=np.uint8)
    v[0, 0], v[0, 16], v[0, 33], v[3, 63] = 1, 2, 3, 4
    u = kv_ref.value_units(v).view(np.uint16)[0]  # [unit][token]
    assert u[0, 0] == 1 | 2 << 4 and u[1, 0] == 3 << 8 and u[15, 3] == 4 << 12
    assert np.count_nonzero(u) == 3


def test_grid_words_by_hand():
    w = kv_ref.grid_words(np.float32([1.0, -2.0, np.nan]), np.float32([8, 0, 8])).view(np.uint32)
    assert [hex(x) for x in w] == ["0x3f800000", "0xc0004800", "0x7fc00000"]


@pytest.mark.parametrize("sym,x,codes,scale,zero", [
    (False, [0.0, 15.0, 7.0, 7.5], [0, 15, 7, 8], 1.0, 0),          # 7.5 to even
    (False, [-8.0, 7.0, 0.0, -0.5], [0, 15, 8, 8], 1.0, 8),         # 7.5 to even
    (False, [4.0, 30.0, 10.0, 2.0], [2, 15, 5, 1], 2.0, 0),         # the range holds 0
    (False, [0.0, 0.0, 0.0, 0.0], [0, 0, 0, 0], 1.0, 0),
    (True, [7.0, -7.0, 2.5, -3.5], [15, 1, 10, 4], 1.0, 8),         # 2.5 and -3.5 to even
    (True, [0.0, 0.0, 0.0, 0.0], [8, 8, 8, 8], 1.0, 8),
])
def test_grids_by_hand(sym, x, codes, scale, zero):
    q, s, z = kv_ref.fit(np.float32([x]), 4, sym)
    assert q[0].tolist() == codes and s[0, 0] == scale and z[0, 0] == zero


def test_scales_are_bf16_and_odd_groups_none():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 64)).astype(np.float32)
    x[3, 40], x[4, 0], x[5, 31], x[5, 30] = np.nan, np.inf, 3.2e38, -3.2e38
    _, s, z = kv_ref.fit(x, 32, False)
    assert np.isnan(s[3, 1]) and np.isnan(s[4, 0]) and np.isnan(s[5, 0]) and np.isnan(s).sum() == 3
    ok = ~np.isnan(s)
    assert ((s[ok].view(np.uint32) & 0xFFFF) == 0).all() and (z[~ok] == 8).all()


@pytest.mark.parametrize("D,g", [(64, 32), (128, 128), (192, 64), (256, 32)])
@pytest.mark.parametrize("sym", [False, True])
def test_same_bytes_as_the_plain_forms(plain, D, g, sym):
    pool = kv_ref.Pool(3, 2, D, 16, g, sym, seed=D)
    k, v, kg, vg, _ = pool.words()
    assert np.array_equal(plain._pack_k(torch.from_numpy(pool.kq)).numpy(), k)
    units = plain._pack_v(torch.from_numpy(pool.vq)).unflatten(-2, (-1, 8)).transpose(-1, -2)
    assert np.array_equal(units.numpy(), v)
    s, z = (torch.from_numpy(t).unsqueeze(-1) for t in (pool.ks, pool.kz))
    assert np.array_equal(plain._grid_words(s, z).transpose(-1, -2).numpy(), kg)
    table = torch.tensor([[2, 0]])
    for name, words, grid in (("k", k, kg), ("v", v, vg)):
        got = plain._values(torch.from_numpy(words), torch.from_numpy(grid), D, table, 16, name == "k")
        q, s, z, there = pool.seq([2, 0], 32, name)
        assert there.all()
        assert np.array_equal(got[0].numpy(), np.repeat(s, g, -1) * (q - np.repeat(z, g, -1)))
        held = plain._held64(dict(k=torch.from_numpy(k), v=torch.from_numpy(v), k_grid=torch.from_numpy(kg), v_grid=torch.from_numpy(vg)),
                             name, table[0], D)
        assert np.array_equal(held.numpy(), np.repeat(s, g, -1).astype(np.float64) * (q - np.repeat(z, g, -1)))
