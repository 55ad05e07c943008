"""What the 4-bit cache's header promises of unusual inputs: finite groups at the end of bf16's range."""
import numpy as np
import pytest

import kv_ref
import post_weight_quantization_21_amd as gq
from gpu_util import host, torch_mod
from test_gpu_kv_cache import ints

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
