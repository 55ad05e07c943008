"""The few-token products (gemv, gemv_gated, moe_layer) at the borders of their paths, types and memory."""
import ctypes

import numpy as np
import pytest

import few_ref as fr
import post_weight_quantization_21_amd as gq
from gpu_util import cuda, host, log, torch_mod
from test_gpu_few_tokens import _acts, _check, _dev, _dt, _experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.load_library()


def _launches(call):
    """The number of kernels that a call launches: the nodes of a graph it is captured into."""
    torch = torch_mod()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph, stream=side):
        call()
    n = ctypes.c_size_t(0)
    get = gq.load_library().hipGraphGetNodes
    get.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]
    assert get(graph.raw_cuda_graph(), None, ctypes.byref(n)) == 0
    return n.value


# One token's experts have one row each: up to GEMV_GATHERS columns the first products gather the order themselves.
@pytest.mark.parametrize("d,E,k,launches", [(gq.GEMV_GATHERS, 4, 2, 6), (gq.GEMV_GATHERS + 32, 4, 2, 7), (2080, 9, 8, 6), (2080, 3, 3, 6)])
def test_moe_one_token_in_a_column_order(oracle_mod, d, E, k, launches):
    torch = torch_mod()
    log(f"moe of one token in a column order: d={d} E={E} k={k}")
    rng = np.random.default_rng(d + k)
    hw, dw = _experts(rng, oracle_mod, E, d, 64, 4, 32, True)
    X, x = _acts(rng, 1, d, "bf16")
    R = cuda((rng.standard_normal((E, d)) * (2 / np.sqrt(d))).astype(np.float32))
    ids, weights = fr.route(x, host(R).astype(np.float64), k, True)
    Y, gi, _ = gq.moe_layer(X, *dw, router=R, top_k=k, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert np.array_equal(host(gi), ids)
    want, bound = fr.moe(x, *hw, ids, weights, "fp32")
    _check(Y, want, bound, "moe")
    assert _launches(lambda: gq.moe_layer(X, *dw, router=R, top_k=k, out_dtype=torch.float32)) == launches


@pytest.mark.parametrize("T,E,k,renorm", [(1, 64, 6, True), (16, 128, 8, True), (16, 128, 8, False), (7, 512, 16, False), (16, 300, 16, True),
                                          (5, 3, 3, False), (16, 1, 1, True), (16, 1, 1, False), (9, 65, 1, False)])
def test_moe_weights_are_rounded_once(oracle_mod, T, E, k, renorm):
    """The softmax is in fp64: a weight is its value rounded to fp32 (half a step; the fp64 sums of 64 products, of at
    most 512 exponentials and of logits of at most 30 are far below the other hundredth)."""
    torch = torch_mod()
    log(f"moe weights T={T} E={E} k={k} renorm={renorm}")
    rng = np.random.default_rng(T + E + k)
    _, dw = _experts(rng, oracle_mod, E, 64, 32, 4, 32, False)
    X, x = _acts(rng, T, 64, "bf16")
    R = cuda((rng.standard_normal((E, 64)) * 0.4).astype(np.float32))
    ids, weights = fr.route(x, host(R).astype(np.float64), k, renorm)
    _, gi, gw = gq.moe_layer(X, *dw, router=R, top_k=k, renormalize=renorm)
    torch.cuda.synchronize()
    assert np.array_equal(host(gi), ids)
    ratio = np.abs(host(gw).astype(np.float64) - weights) / (1.01 * fr.U * weights)
    log(f"  worst error over the bound {ratio.max():.3f}")
    assert (ratio <= 1).all()


@pytest.mark.parametrize("E,low,high", [(2, 0, 1), (64, 3, 60), (300, 5, 299), (512, 130, 448)])
def test_moe_router_ranks_by_every_bit(oracle_mod, E, low, high):
    """Logits of 1 and 1 + 2^-48, both exact in the router's fp64 sum: the larger comes first whatever its index."""
    torch = torch_mod()
    rng = np.random.default_rng(E)
    _, dw = _experts(rng, oracle_mod, E, 64, 32, 4, 32, False)
    X = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    X[0, 0], X[0, 1] = 1.0, 2.0 ** -24
    for first, second in ((high, low), (low, high)):
        R = torch.full((E, 64), -1.0, device="cuda")
        R[[low, high], 0] = 1.0
        R[[low, high], 1] = 0.0
        R[first, 1] = 2.0 ** -24
        _, ids, _ = gq.moe_layer(X, *dw, router=R, top_k=2)
        assert ids[0].tolist() == [first, second]
    R[first, 1] = 0.0  # equal: the lower index first
    _, ids, _ = gq.moe_layer(X, *dw, router=R, top_k=2)
    assert ids[0].tolist() == [low, high]


# (M, d_out, d_in, bits, group, out): a value per token as large as bf16 holds (8 bits: 2^119), whose sums the
# definition leaves finite
@pytest.mark.parametrize("M,d_out,d_in,bits,group,out", [
    (1, 40, 160, 2, 32, "fp32"), (3, 40, 512, 2, 128, "bf16"), (2, 33, 160, 3, 0, "fp32"), (16, 20, 640, 3, 32, "bf16"),
    (1, 40, 160, 4, 32, "bf16"), (16, 70, 1024, 4, 128, "fp32"), (2, 40, 160, 8, 32, "fp32"), (5, 40, 1024, 8, 128, "bf16")])
def test_gemv_of_the_largest_bf16_activations(oracle_mod, M, d_out, d_in, bits, group, out):
    torch = torch_mod()
    log(f"gemv of large activations M={M} {d_out}x{d_in} {bits} bits g={group} -> {out}")
    rng = np.random.default_rng(d_in + bits)
    w = fr.make_packed(rng, oracle_mod, d_out, d_in, bits, group)
    X, _ = _acts(rng, M, d_in, "bf16")
    for m in range(M):
        X[m, int(rng.integers(d_in))] = float(rng.choice([-1, 1])) * (2.0 ** 119 if bits == 8 else torch.finfo(torch.bfloat16).max)
    x = host(X.float()).astype(np.float64)
    want, bound = fr.product(x, w)
    assert np.abs(want).max() < 2.0 ** 127
    _check(gq.gemv(X, _dev(w), out_dtype=_dt(out)), want, fr.rounded(want, bound, out), "large activations")


def test_gated_of_very_negative_gates(oracle_mod):
    """silu(g) u where exp(-g) is past fp32's range, and silu(g) alone near or below its smallest numbers: g from -86
    to -200, u of 2^100."""
    torch = torch_mod()
    d_out, d_in, U0 = 115, 32, 2.0 ** 100
    gate, up = (dict(q=np.full((d_out, d_in), 0, dtype=np.uint8), scales=np.ones((d_out, 1), dtype=np.float32),
                     zeros=np.zeros((d_out, 1), dtype=np.float32), kperm=None, bits=8, group=0) for _ in range(2))
    gate["q"][:, 1] = 86 + np.arange(d_out)  # times x = -1
    up["q"][:, 0] = 1
    up["scales"][:] = U0
    for w in (gate, up):
        w["packed"] = oracle_mod.pack_codes(w["q"], 8)
    for dt in ("bf16", "fp16"):
        X = torch.zeros(2, d_in, dtype=_dt(dt), device="cuda")
        X[:, 0], X[:, 1], X[1, 0] = 1.0, -1.0, -1.0
        H = host(gq.gemv_gated(X, _dev(gate), _dev(up), out_dtype=torch.float32)).astype(np.float64)
        g = -(86.0 + np.arange(d_out))
        want = g * np.exp(g) / (1 + np.exp(g)) * U0 * np.array([[1.0], [-1.0]])
        # the sums are exact; two exponentials, three products: 8 ulp of fp32 as for the ordinary values
        bound = 16 * fr.U * np.abs(want) + 2.0 ** -149
        log(f"  worst err/bound {(np.abs(H - want) / bound).max():.3g}")
        assert (np.abs(H - want) <= bound).all()


def test_few_tokens_results_between_the_rows_of_x(oracle_mod):
    """X and the results as columns of one tensor, next to each other but apart: allowed, and X stays as it was."""
    torch = torch_mod()
    rng = np.random.default_rng(21)
    d, M, E = 128, 5, 4
    w = _dev(fr.make_packed(rng, oracle_mod, d, d, 4, 32))
    _, dw = _experts(rng, oracle_mod, E, d, d, 4, 32, False)
    X, _ = _acts(rng, M, d, "bf16")
    ids = torch.arange(M, dtype=torch.int32, device="cuda").remainder(E).view(M, 1)
    weights = torch.ones(M, 1, device="cuda")
    buf = torch.zeros(M, 4 * d, dtype=torch.bfloat16, device="cuda")
    x, y, h, z = buf.split(d, dim=1)
    x.copy_(X)
    gq.gemv(x, w, Y=y)
    gq.gemv_gated(x, w, w, H=h)
    gq.moe_layer(x, *dw, ids=ids, weights=weights, Y=z)
    assert torch.equal(x, X) and torch.equal(y, gq.gemv(X, w)) and torch.equal(h, gq.gemv_gated(X, w, w))
    assert torch.equal(z, gq.moe_layer(X, *dw, ids=ids, weights=weights)[0])
    for call in (lambda: gq.gemv(X, w, Y=X), lambda: gq.gemv_gated(X, w, w, H=X), lambda: gq.moe_layer(X, *dw, ids=ids, weights=weights, Y=X)):
        with pytest.raises(gq.GptqError) as ei:
            call()
        assert ei.value.status == gq.ERR_INVALID_ARG
