"""The plan of moe_linear, compiled on its own: the sizes that the GPU tests run
reach every kernel instance that it can choose (no GPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests._lib import ROOT
from tests.linear_plan_shapes import PRODUCTS

SMS = 152
SHIM = """
#include "linear_plan.h"
extern "C" void plans(int n, const int* tnk, int sms, int* out) {
  for (int i = 0; i < n; ++i) {
    const moe::LinearPlan p = moe::linear_plan(tnk[3 * i], tnk[3 * i + 1], (tnk[3 * i + 2] + 63) / 64, sms);
    out[2 * i] = p.pair ? -p.nt : p.nt;
    out[2 * i + 1] = p.splits;
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                           os.path.join(ROOT, "int4_routed_expert_moe_gb300", "csrc"), str(d / "shim.cpp"), "-o",
                           str(d / "shim.so")])
    lib = ctypes.CDLL(str(d / "shim.so"))

    def call(sizes):
        a = np.ascontiguousarray(sizes, dtype=np.int32).reshape(-1, 3)
        out = np.empty((len(a), 2), np.int32)
        lib.plans(len(a), a.ctypes.data_as(ctypes.c_void_p), SMS, out.ctypes.data_as(ctypes.c_void_p))
        return [tuple(int(v) for v in p) for p in out]
    return call


def test_sizes_run_on_the_instance_they_are_listed_for(plans):
    for plan, sizes in PRODUCTS.items():
        assert plans(sizes) == [plan] * len(sizes), plan


def test_every_reachable_instance_is_listed(plans):
    rng = np.random.default_rng(0)
    spread = lambda lo, hi, n: np.exp(rng.uniform(np.log(lo), np.log(hi), n)).round()
    n = 400_000
    T = np.concatenate([spread(17, 1 << 20, n // 4), spread(17, 4096, n - n // 4)])
    assert set(plans(np.stack([T, spread(1, 65536, n), spread(1, 8192, n) * 8], 1))) == set(PRODUCTS)


def test_splits_never_exceed_the_steps_or_a_wave(plans):
    rng = np.random.default_rng(1)
    sizes = np.stack([rng.integers(17, 3000, 20000), rng.integers(1, 9000, 20000), rng.integers(1, 600, 20000) * 8], 1)
    for (T, N, K), (nt, s) in zip(sizes, plans(sizes)):
        if s > 1:
            assert nt > 0 and s <= -(-K // 64) and -(-T // 128) * -(-N // nt) * s <= SMS


def test_strided_sizes_run_on_the_pair_kernels(plans):
    from tests.test_gpu_linear_plans import STRIDED
    for plan, sizes in STRIDED.items():
        assert plans(sizes) == [plan] * len(sizes), plan
