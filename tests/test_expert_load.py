"""What the mixture's kernels are planned for: the expected number of distinct experts and the tokens that share one."""
import ctypes
import itertools
import math
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_weight_quantization_21_amd", "csrc")


@pytest.fixture(scope="module")
def expert_load(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("g++ is not available")
    d = tmp_path_factory.mktemp("load")
    (d / "load.cpp").write_text('#include "expert_load.h"\n'
                                'extern "C" double experts(long t, int e, int k) { return gptq::expert_load(t, e, k).experts; }\n'
                                'extern "C" int rows(long t, int e, int k) { return gptq::expert_load(t, e, k).rows; }\n')
    subprocess.run([cc, "-std=c++17", "-O2", "-shared", "-fPIC", f"-I{CSRC}", str(d / "load.cpp"), "-o", str(d / "load.so")], check=True)
    lib = ctypes.CDLL(str(d / "load.so"))
    lib.experts.restype = ctypes.c_double
    lib.experts.argtypes = lib.rows.argtypes = [ctypes.c_long, ctypes.c_int, ctypes.c_int]
    return lib


def test_every_size(expert_load):
    for E, k in itertools.product(range(1, 513), range(1, 17)):
        if k > E:
            continue
        assert expert_load.rows(1, E, k) == 1 and abs(expert_load.experts(1, E, k) - k) < 1e-9  # one token's are distinct
        if k == E:
            assert all(expert_load.rows(t, E, k) == t for t in range(1, 17))
        for t in range(1, 17):
            n, r = expert_load.experts(t, E, k), expert_load.rows(t, E, k)
            assert k - 1e-9 < n < min(E, t * k) + 1e-9
            assert 1 <= r <= t and r * n > t * k * (1 - 1e-6) and (r - 1) * n < t * k


@pytest.mark.parametrize("E,k,t", [(4, 2, 3), (5, 1, 4), (6, 3, 2)])
def test_expected_experts_by_counting(expert_load, E, k, t):
    choices = list(itertools.combinations(range(E), k))
    total = sum(len(set().union(*c)) for c in itertools.product(choices, repeat=t))
    want = total / math.comb(E, k) ** t
    assert abs(expert_load.experts(t, E, k) - want) < 1e-9
    assert expert_load.rows(t, E, k) == min(t, math.ceil(t * k / want - 1e-9))
