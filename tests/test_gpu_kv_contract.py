"""What the 4-bit cache's header promises of unusual inputs: finite groups at the end of bf16's range, bad
queries beside hidden tokens."""
import numpy as np
import pytest

import kv_ref
import post_weight_quantization_21_amd as gq
from gpu_util import host, torch_mod
from test_gpu_kv_cache import ints, make_queries, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.load_library()


# ---- append ---------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("heads", [2, 300])  # token by token, and in staged blocks
@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("D,g", [(64, 32), (64, 64), (128, 32), (128, 128), (192, 64), (192, 192), (256, 64), (256, 256)])
def test_append_of_finite_groups_whose_sum_is_not(D, g, sym, heads):
    """Runs of eight values of one sign near bf16's end, next to runs of the other: every value and the spread are finite (or, of
    symmetric grids, the largest value), while sums of neighbours reach both infinities."""
    torch = torch_mod()
    T, page = 33, 16
    pool = kv_ref.Pool(4, heads, D, page, g, sym, seed=D)
    cache = kv_ref.cuda_cache(gq, torch, pool)
    rng = np.random.default_rng(D + g)
    sign = np.where(np.arange(D) // 8 % 2, -1.0, 1.0)
    # spreads up to 2^127.9; symmetric grids take every value that bf16 has
    top = 3.38e38 if sym else 1.69e38
    x = sign * top * rng.uniform(0.6, 1.0, (T, heads, D))
    x[5] *= -1
    x[6, :, ::2] = 0
    x[7, :, g // 2:] *= 2.0 ** -120
    x[8:12] = sign * top * np.array([1.0, 0.5, 2.0 ** -20, 0.75])[:, None, None]
    x = torch.from_numpy(x).to(torch.bfloat16)
    bad = x.clone()
    bad[20, 0, 3], bad[21, 1, g - 1], bad[22, 0, 0], bad[23, 1, 8] = float("nan"), float("inf"), -float("inf"), float("-nan")
    K, V = x, bad
    k, v = gq.kv_append(K.cuda(), V.cuda(), cache, ints([[1, 3, 0]]), ints([T]), values=True)
    for side, a, got in (("k", K, k), ("v", V, v)):
        q, s, z = kv_ref.fit(a.float().numpy(), g, sym)
        assert np.isnan(s).sum() == (4 if side == "v" else 0)
        for name, val in (("q", q), ("s", s), ("z", z)):
            for t in range(T):
                getattr(pool, side + name)[[1, 3, 0][t // page], :, t % page] = val[t]
        want = torch.from_numpy((np.repeat(s, g, -1) * (q - np.repeat(z, g, -1))).astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got.cpu()), torch.nan_to_num(want))
    for t in range(T):
        pool.weight[[1, 3, 0][t // page], :, t % page] = 0
    for name, want, have in zip("k v k_grid v_grid weight".split(), pool.words(), cache.tensors):
        assert np.array_equal(host(have), want), name


# ---- weights --------------------------------------------------------------------------------------------------------

#          lens              n   Hq  Hkv D    g   page
WEIGHED = [([90, 50], 3, 4, 2, 64, 32, 16),
           ([700, 1300, 9], 4, 8, 2, 128, 128, 64),   # split over workgroups; four new tokens
           ([333, 40, 16], 16, 32, 2, 64, 64, 32),    # 256 columns: several passes over the tokens
           ([260], 16, 3, 1, 192, 64, 16),
           ([515, 2], 5, 7, 1, 256, 0, 128)]          # two tokens of five new ones


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("case", WEIGHED, ids=lambda c: "-".join(str(x) for x in c if not isinstance(x, list)))
def test_weights_of_tokens_that_a_bad_query_does_not_see(case, decay):
    """A query that is no number makes the weights of all that it sees no numbers, of its kv head alone; new tokens behind it,
    which it does not see, get what the others give them."""
    torch = torch_mod()
    lens, n, Hq, H, D, g, page = case
    B = len(lens)
    width = -(-max(lens) // page) + 1
    pool = kv_ref.Pool(B * width + 1, H, D, page, g, False, seed=D)
    table = tables(np.random.default_rng(n + D), B * width + 1, B, width)
    q, q64 = make_queries((B, n, Hq, D), "bf16", 5)
    bad = q.clone()
    at = n // 2 - 1  # the query's token; those behind it are hidden from it
    bad[0, at, 0, 5], bad[B - 1, 0, Hq - 1, D - 1] = float("nan"), float("inf")
    cache = kv_ref.cuda_cache(gq, torch, pool)
    o = gq.kv_attention(bad.cuda(), cache, ints(table), ints(lens), decay=decay)
    _, _, _, weight, wtol = kv_ref.attention(pool, q64, table, lens, D ** -0.5, "bf16", decay)
    got = host(cache.weight).astype(np.float64)
    none = np.zeros(got.shape, dtype=bool)
    for b, i, h in ((0, at, 0), (B - 1, 0, H - 1)):
        slot = np.arange(max(0, lens[b] - n + 1 + i))
        none[table[b, slot // page], h, slot % page] = True
        seen = len(slot) > 0
        row = o[b, i, 0 if h == 0 and i == at else Hq - 1].float().cpu()
        assert bool(torch.isfinite(row).all()) == (not seen)
    assert np.isnan(got[none]).all()
    assert not np.isnan(got[~none]).any()
    assert (np.abs(got - weight)[~none] <= wtol[~none]).all()
