"""The balance loss's plan, compiled on its own: the border cases of the GPU tests sit on its borders (no GPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests._lib import ROOT
from tests.balance_plan_shapes import BORDERS

SHIM = """
#include "balance_plan.h"
extern "C" void plans(int n, const int* a, int back, int* out) {
  for (int i = 0; i < n; ++i, a += 4) {
    const moe::BalancePlan p = moe::balance_plan(a[0], a[1], a[3], back);
    out[5 * i] = p.chunk;
    out[5 * i + 1] = p.chunks;
    out[5 * i + 2] = p.fused ? 1 : 2;
    out[5 * i + 3] = moe::sequences_of(moe::lanes_of(a[1]), moe::values_of(a[1]));
    out[5 * i + 4] = moe::max_chunks(a[1]);
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

    def call(cases, back=False):
        a = np.ascontiguousarray(cases, dtype=np.int32).reshape(-1, 4)
        out = np.empty((len(a), 5), np.int32)
        lib.plans(len(a), a.ctypes.data_as(ctypes.c_void_p), int(back), out.ctypes.data_as(ctypes.c_void_p))
        return [tuple(int(v) for v in p) for p in out]
    return call


def test_border_cases_sit_on_the_borders(plans):
    for case, (_, chunks, launches, per_pass, _) in zip(BORDERS, plans(list(BORDERS))):
        assert BORDERS[case] == (chunks, launches, case[3] > per_pass), (case, chunks, launches, per_pass)


def test_each_border_is_crossed(plans):
    # One more token or sequence than the largest batch of one block, for each way of sharing a token.
    for E in (64, 128, 256, 512):
        one = max(c[0] for c, p in BORDERS.items() if c[1] == E and c[3] == 16 and p[0] == 1)
        assert plans([(one + 1, E, 1, 16)])[0][1] > 1 and (one + 1, E) in {c[:2] for c in BORDERS}, E
    assert plans([(288, 64, 1, 16)])[0][1] == 1 and plans([(288, 64, 1, 17)])[0][1] > 1


def test_a_plan_covers_its_tokens_and_fits_the_workspace(plans):
    rng = np.random.default_rng(0)
    T = np.exp(rng.uniform(0, np.log(1 << 27), 5000)).astype(int)
    cases = np.stack([T, rng.integers(1, 1025, 5000), np.ones(5000, int), rng.integers(1, 40, 5000)], 1)
    for back in (False, True):
        for c, (chunk, chunks, launches, _, most) in zip(cases, plans(cases, back)):
            assert chunk * chunks >= c[0] > chunk * (chunks - 1) and (back or chunks <= max(1, min(-(-c[0] // 32), most)))
            assert (launches == 1) == (chunks * c[1] <= 40960)
