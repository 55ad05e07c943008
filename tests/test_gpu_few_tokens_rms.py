"""The few-token products on random data: the root mean square of their errors, with fp32 results."""
import numpy as np
import pytest

import few_ref as fr
import few_rms
import post_weight_quantization_21_amd as gq
from gpu_util import cuda, host, log, torch_mod
from test_gpu_few_tokens import GEMV, MOE, _acts, _dev, _dt, _experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.load_library()


def _within(got, want, var, out):
    r = few_rms.rms(host(got.float()).astype(np.float64), want, var, out)
    log(f"  {out}: root mean square of error / sigma {r:.3f}")
    assert r <= 1


@pytest.mark.parametrize("M,d_out,d_in,bits,group,dt,perm", [c[:6] + (c[7],) for c in GEMV])
def test_gemv_and_gated_errors(oracle_mod, M, d_out, d_in, bits, group, dt, perm):
    log(f"errors M={M} {d_out}x{d_in} {bits} bits g={group} {dt} perm={perm}")
    rng = np.random.default_rng(M + 7 * d_in + bits)
    gate, up = (fr.make_packed(rng, oracle_mod, d_out, d_in, bits, group, perm) for _ in range(2))
    up["kperm"] = gate["kperm"]
    X, x = _acts(rng, M, d_in, dt)
    dg = _dev(gate)
    du = gq.packed_weight(cuda(up["packed"].view(np.int32)), cuda(up["scales"]), cuda(up["zeros"]), bits, group, kperm=dg.kperm)
    (g, var_g), (u, var_u) = few_rms.product(x, gate), few_rms.product(x, up)
    for out in ("fp32", dt):
        _within(gq.gemv(X, dg, out_dtype=_dt(out)), g, var_g, out)
        _within(gq.gemv_gated(X, dg, du, out_dtype=_dt(out)), *few_rms.silu_mul(g, var_g, u, var_u), out)


@pytest.mark.parametrize("T,d,ff,E,k,bits,group,dt,perm", [c[:8] + (c[9],) for c in MOE])
def test_moe_errors(oracle_mod, T, d, ff, E, k, bits, group, dt, perm):
    log(f"errors of moe T={T} d={d} ff={ff} E={E} k={k} {bits} bits g={group} {dt} perm={perm}")
    rng = np.random.default_rng(T * 3 + d + E)
    hw, dw = _experts(rng, oracle_mod, E, d, ff, bits, group, perm)
    X, x = _acts(rng, T, d, dt)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = rng.uniform(0.1, 1, size=ids.shape).astype(np.float32)
    for out in ("fp32", dt):
        Y = gq.moe_layer(X, *dw, ids=cuda(ids), weights=cuda(weights), out_dtype=_dt(out))[0]
        _within(Y, *few_rms.moe(x, *hw, ids, weights.astype(np.float64), 3 if out == "fp32" else 2), out)
