"""Host-side argument checks of the scored-routing and FP8 entry points (no GPU)."""
import ctypes

import pytest

from tests._lib import binding

moe = binding()
lib = moe._lib


def _route(cfg, ltype=0, ld=16, T=4, E=16, k=2):
    return lib.moe_route_scored(cfg, None, ltype, ld, T, E, k, None, None, None, None, None)


def test_route_scored_arguments():
    ok = moe.moe_route_config()
    assert _route(None) == moe.MOE_ERR_ARG
    assert _route(ok, T=0) == moe.MOE_OK
    assert _route(ok) == moe.MOE_ERR_ARG  # NULL pointers
    assert "NULL" in moe.moe_last_error()
    for kw in (dict(k=0), dict(k=17), dict(E=0), dict(E=1025, ld=2000), dict(T=-1), dict(ld=15), dict(ltype=2),
               dict(k=33, E=64, ld=64)):
        assert _route(ok, **{"T": 0, **kw}) == moe.MOE_ERR_ARG, kw
    for kw in (dict(n_groups=3), dict(n_groups=0), dict(n_groups=64), dict(n_groups=4, top_groups=0),
               dict(n_groups=4, top_groups=5), dict(n_groups=16, top_groups=1), dict(scale=float("inf"))):
        assert _route(moe.moe_route_config(**kw), T=0) == moe.MOE_ERR_ARG, kw
    bad = moe.moe_route_config()
    for field in ("score", "group_rank"):
        c = moe.moe_route_config()
        setattr(c, field, 2)
        assert _route(c, T=0) == moe.MOE_ERR_ARG
    with pytest.raises(KeyError):
        moe.moe_route_config(score="relu")
    assert ctypes.sizeof(bad) == 24


def test_fp8_arguments():
    q = lib.moe_quantize_fp8
    assert q(None, 0, 64, 1, None, None, None) == moe.MOE_OK
    assert q(None, 4, 64, 1, None, None, None) == moe.MOE_ERR_ARG
    for rows, cols, br in ((0, 40, 1), (0, 0, 1), (-1, 64, 1), (0, 64, 3), (0, 65552, 1), (1 << 30, 64, 1),
                           (65535 * 128 + 1, 64, 128)):
        assert q(None, rows, cols, br, None, None, None) == moe.MOE_ERR_ARG, (rows, cols, br)
    m = lambda T, N, K: lib.moe_matmul_fp8(None, None, T, None, None, N, K, None, None, 0, None)
    assert m(0, 8, 16) == moe.MOE_OK
    for a in ((4, 8, 16), (0, 0, 16), (0, 8, 8), (0, 8, 24), (-1, 8, 16), ((1 << 20) + 1, 8, 16), (0, 65537, 16),
              (0, 8, 65552)):
        assert m(*a) == moe.MOE_ERR_ARG, a
    s = lambda T, H, I: lib.moe_shared_forward_fp8(None, T, H, I, *[None] * 8, 0, None)
    assert s(0, 64, 64) == moe.MOE_OK
    for a in ((1, 64, 64), (0, 96, 64), (0, 64, 0), (-1, 64, 64), (0, 64, 65600)):
        assert s(*a) == moe.MOE_ERR_ARG, a


def test_fp8_workspace_sizes():
    assert moe.moe_matmul_fp8_workspace_bytes(4, 64, 24) == 0
    assert moe.moe_matmul_fp8_workspace_bytes(4, 64, 128) >= 256
    assert moe.moe_shared_fp8_workspace_bytes(4, 96, 64) == 0
    T, H, Is = 100, 512, 320
    assert moe.moe_shared_fp8_workspace_bytes(T, H, Is) >= 256 + T * (H + Is) + T * (4 + 3) * 4
    # A workspace for T tokens serves any smaller batch.
    for H, Is in ((64, 64), (512, 320), (64, 4096)):
        sizes = [moe.moe_shared_fp8_workspace_bytes(T, H, Is) for T in range(0, 70)]
        assert sizes == sorted(sizes)
