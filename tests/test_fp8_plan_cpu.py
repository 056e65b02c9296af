"""The plan of the FP8 product, compiled on its own: the sizes that the GPU tests
run reach every kernel instance that it can choose (no GPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests._lib import ROOT
from tests.fp8_plan_shapes import GATE_UPS, PRODUCTS

SMS = 152
SHIM = """
#include "fp8_plan.h"
extern "C" void plans(int n, const int* tnk, int sms, int gateup, int* out) {
  for (int i = 0; i < n; ++i) {
    const moe::Plan p = moe::plan_of(tnk[3 * i], tnk[3 * i + 1], (tnk[3 * i + 2] + 127) / 128, sms, gateup != 0);
    out[2 * i] = p.nt;
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

    def call(sizes, gateup):
        a = np.ascontiguousarray(sizes, dtype=np.int32).reshape(-1, 3)
        out = np.empty((len(a), 2), np.int32)
        lib.plans(len(a), a.ctypes.data_as(ctypes.c_void_p), SMS, int(gateup), out.ctypes.data_as(ctypes.c_void_p))
        return [tuple(int(v) for v in p) for p in out]
    return call


@pytest.mark.parametrize("table,gateup", [(PRODUCTS, False), (GATE_UPS, True)], ids=["product", "gate_up"])
def test_sizes_run_on_the_instance_they_are_listed_for(plans, table, gateup):
    for plan, sizes in table.items():
        assert plans(sizes, gateup) == [plan] * len(sizes), plan


@pytest.mark.parametrize("table,gateup", [(PRODUCTS, False), (GATE_UPS, True)], ids=["product", "gate_up"])
def test_every_reachable_instance_is_listed(plans, table, gateup):
    rng = np.random.default_rng(0)
    spread = lambda lo, hi, n: np.exp(rng.uniform(np.log(lo), np.log(hi), n)).round()
    n, unit = 400_000, 64 if gateup else 1
    T = np.concatenate([spread(17, 1 << 20, n // 4), spread(17, 4096, n - n // 4)])
    N = spread(1, 65536 // unit, n) * unit
    K = spread(1, 1024, n) * 64 if gateup else spread(1, 4096, n) * 16
    assert set(plans(np.stack([T, N, K], 1), gateup)) == set(table)
