"""gemv_gated and moe_layer on layers of small integers, where they are exact but for the result's rounding."""
import numpy as np
import pytest

import few_exact as fx
import few_ref as fr
import post_weight_quantization_21_amd as gq
from gpu_util import cuda, host, log, torch_mod
from test_gpu_few_tokens import _dev, _dt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.load_library()


def _pair(gate, up):
    dg = _dev(gate)
    return dg, gq.packed_weight(cuda(up["packed"].view(np.int32)), cuda(up["scales"]), cuda(up["zeros"]), up["bits"], up["group"], kperm=dg.kperm)


def _equal(got, want, out):
    """want is exact in fp32; the result is it, rounded to nearest even."""
    torch = torch_mod()
    want = cuda(want.astype(np.float32)).to(_dt(out))
    assert torch.equal(got, want), f"{(got != want).double().mean().item():.3g} of the values differ"


# (M, d_out, d_in, bits, group, dt, out, perm)
GATED = [
    (1, 1, 32, 4, 0, "bf16", "fp32", False),
    (1, 100, 4096, 4, 128, "bf16", "fp32", True),      # a column order gathered by the product, the most columns
    (1, 100, 4128, 4, 96, "fp16", "fp32", True),       # ... and prepared by a kernel of its own
    (5, 130, 1056, 8, 32, "bf16", "fp32", True),
    (16, 70, 512, 3, 32, "fp16", "bf16", True),
    (3, 200, 2720, 8, 0, "bf16", "fp16", False),
    (16, 48, 16384, 4, 128, "bf16", "fp32", False),    # several phases
    (16, 40, 12288, 2, 64, "fp16", "fp32", True),      # ... of prepared activations, groups inside a step
    (9, 33, 20480, 3, 32, "bf16", "fp32", True),
    (16, 33, 8192, 8, 256, "fp16", "fp32", False),
    (8, 4200, 2048, 4, 64, "fp16", "fp32", False),
    (2, 31, 160, 2, 32, "bf16", "bf16", False),
    (7, 50, 416, 3, 0, "bf16", "fp32", False),
]


@pytest.mark.parametrize("M,d_out,d_in,bits,group,dt,out,perm", GATED)
def test_gated_of_integers(oracle_mod, M, d_out, d_in, bits, group, dt, out, perm):
    log(f"gated of integers M={M} {d_out}x{d_in} {bits} bits g={group} {dt}->{out} perm={perm}")
    rng = np.random.default_rng(M + d_in + bits)
    gate, up = fx.gate_and_up(rng, oracle_mod, (d_out, d_in), bits, group, perm, True)
    x = fx.acts(rng, M, d_in)
    want = fx.gated(x, gate, up)
    _equal(gq.gemv_gated(cuda(x.astype(np.float32)).to(_dt(dt)), *_pair(gate, up), out_dtype=_dt(out)), want, out)


# (T, d, ff, E, k, bits, group, dt, out, perm): for an fp32 result h takes three bf16 values (one token
# has few of h), else no more than two
MOE = [
    (1, 64, 320, 1, 1, 4, 0, "bf16", "fp32", False),
    (1, 4096, 288, 4, 2, 8, 32, "fp16", "fp32", True),    # one token gathers the order itself: the most columns
    (1, 4128, 288, 4, 2, 4, 96, "bf16", "fp32", True),    # ... and has it prepared
    (3, 160, 736, 5, 3, 4, 32, "bf16", "fp32", False),
    (16, 256, 640, 12, 3, 4, 128, "bf16", "fp32", False),
    (16, 4096, 224, 2, 2, 4, 32, "bf16", "fp32", False),   # every expert all tokens: phases of the first products
    (16, 512, 7168, 2, 1, 4, 64, "fp16", "fp32", True),    # ... and of the second, in three pieces
    (16, 1024, 640, 3, 2, 2, 32, "bf16", "fp32", True),
    (9, 128, 5120, 3, 2, 3, 128, "fp16", "fp32", False),
    (16, 512, 1056, 3, 3, 3, 32, "bf16", "fp32", True),
    (5, 352, 2560, 4, 2, 8, 0, "fp16", "fp32", True),
    (16, 256, 512, 12, 3, 4, 128, "bf16", "bf16", False),
    (7, 512, 7168, 2, 1, 4, 64, "fp16", "fp16", True),
    (16, 128, 640, 3, 2, 2, 32, "fp16", "bf16", True),
    (4, 352, 2560, 4, 2, 8, 32, "bf16", "bf16", False),
    (2, 96, 1152, 4, 2, 3, 96, "bf16", "fp16", False),
]


@pytest.mark.parametrize("T,d,ff,E,k,bits,group,dt,out,perm", MOE)
def test_moe_of_integers(oracle_mod, T, d, ff, E, k, bits, group, dt, out, perm):
    log(f"moe of integers T={T} d={d} ff={ff} E={E} k={k} {bits} bits g={group} {dt}->{out} perm={perm}")
    rng = np.random.default_rng(T + d + ff + bits)
    gate, up, down = fx.experts(rng, oracle_mod, E, d, ff, bits, group, perm, out == "fp32")
    if out == "fp16":  # its range
        down["scales"] = down["scales"] / np.float32(64)
    x = fx.acts(rng, T, d)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = rng.choice(np.array([1.0, 2.0], dtype=np.float32), size=ids.shape)
    want, pieces = fx.moe(x, gate, up, down, ids, weights.astype(np.float64))
    assert pieces >= (3 if T > 1 else 2) if out == "fp32" else pieces <= 2
    got, _, _ = gq.moe_layer(cuda(x.astype(np.float32)).to(_dt(dt)), *_pair(gate, up), _dev(down), ids=cuda(ids), weights=cuda(weights),
                             out_dtype=_dt(out))
    _equal(got, want, out)


# h of more than 17 bits with 16-bit results: enough of them for a rounding to fall to the other side
@pytest.mark.parametrize("T,d,ff,E,k,bits,group,dt,out,perm", [
    (16, 4096, 640, 2, 2, 3, 32, "bf16", "bf16", False),
    (16, 4096, 640, 2, 2, 8, 128, "fp16", "fp16", True),
    (16, 4096, 1152, 2, 1, 2, 64, "bf16", "fp16", True),
])
def test_moe_of_large_integers_with_16_bit_results(oracle_mod, T, d, ff, E, k, bits, group, dt, out, perm):
    log(f"moe of large integers T={T} d={d} ff={ff} E={E} k={k} {bits} bits g={group} {dt}->{out} perm={perm}")
    rng = np.random.default_rng(T + d + ff + bits)
    gate, up, down = fx.experts(rng, oracle_mod, E, d, ff, bits, group, perm, True)
    if out == "fp16":
        down["scales"] = down["scales"] / np.float32(512)
    x = fx.acts(rng, T, d)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = rng.choice(np.array([1.0, 2.0], dtype=np.float32), size=ids.shape)
    want, pieces = fx.moe(x, gate, up, down, ids, weights.astype(np.float64))
    assert pieces == 3
    got, _, _ = gq.moe_layer(cuda(x.astype(np.float32)).to(_dt(dt)), *_pair(gate, up), _dev(down), ids=cuda(ids), weights=cuda(weights),
                             out_dtype=_dt(out))
    _equal(got, want, out)


@pytest.mark.parametrize("bits,dt", [(4, "bf16"), (8, "fp16")])
def test_moe_rows_of_every_size(oracle_mod, bits, dt):
    """Each token's h is scaled by a power of two of its own: up matrices of 2^-60 to 2^60, tokens whose h is zero."""
    torch = torch_mod()
    rng = np.random.default_rng(bits)
    E, T, d, ff = 3, 9, 128, 640
    gate, up, down = fx.experts(rng, oracle_mod, E, d, ff, bits, 32, False, True)
    x = fx.acts(rng, T, d)
    ids = np.arange(T, dtype=np.int32).reshape(T, 1) % E
    weights = np.ones((T, 1), dtype=np.float32)
    want, _ = fx.moe(x, gate, up, down, ids, weights.astype(np.float64))
    X = cuda(x.astype(np.float32)).to(_dt(dt))
    for exps in ((-60, 0, 60), (60, -100, 3), (-126 + 40, 80, 0)):
        scaled = dict(up, scales=up["scales"] * np.float32(2) ** np.array(exps, dtype=np.float32)[:, None, None])
        got = gq.moe_layer(X, *_pair(gate, scaled), _dev(down), ids=cuda(ids), weights=cuda(weights), out_dtype=torch.float32)[0]
        _equal(got, want * 2.0 ** np.array(exps, dtype=np.float64)[ids], "fp32")
    X[4] = 0
    got = gq.moe_layer(X, *_pair(gate, up), _dev(down), ids=cuda(ids), weights=cuda(weights), out_dtype=torch.float32)[0]
    want[4] = 0
    _equal(got, want, "fp32")


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_moe_small_hidden_values_beside_large_ones(oracle_mod, bits):
    """One hidden value of 2^20 units that the second product does not use (its codes are the zero point), beside values
    from 2^-20 to 2^20 of its units: what a value loses is at most 2^-24 of itself or 2^-39 of the largest."""
    torch = torch_mod()
    rng = np.random.default_rng(bits)
    d, ff = 64, 64
    gate, up = fx.gate_and_up(rng, oracle_mod, (1, ff, d), bits, 32, False, False)
    up["scales"] = up["scales"] * (2.0 ** np.concatenate([[20], rng.integers(-20, 12, size=ff - 1)])).astype(np.float32)[None, :, None]
    x = fx.acts(rng, 3, d)
    h = np.stack([fr.product(x, gate, 0)[0], fr.product(x, up, 0)[0]]).prod(axis=0)
    # the second product picks one hidden value per row: row k is value k, and the large one is used by no row but its own
    down = dict(q=np.zeros((1, ff, ff), dtype=np.uint8), scales=np.ones((1, ff, 2), dtype=np.float32), zeros=np.ones((1, ff, 2), dtype=np.float32),
                kperm=None, bits=bits, group=32)
    down["q"][:] = 1
    down["q"][0, np.arange(ff), np.arange(ff)] = 2
    fx.pack(down, oracle_mod)
    got = gq.moe_layer(cuda(x.astype(np.float32)).bfloat16(), *_pair(gate, up), _dev(down), ids=torch.zeros(3, 1, dtype=torch.int32, device="cuda"),
                       weights=torch.ones(3, 1, device="cuda"), out_dtype=torch.float32)[0]
    err = np.abs(got.cpu().numpy().astype(np.float64) - h)
    bound = np.maximum(2.0 ** -24 * np.abs(h), 2.0 ** -39 * np.abs(h).max(axis=1, keepdims=True))
    log(f"  worst error / bound {np.max(err / np.maximum(bound, 1e-300)):.3f}")
    assert (err <= bound).all()
