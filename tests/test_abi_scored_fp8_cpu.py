"""Host-side argument checks of the scored-routing and FP8 entry points (no GPU)."""
import ctypes

import pytest
import torch

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


def test_shared_fp8_weight_and_scale_shapes():
    # Checked before any pointer is taken, so tensors of the host do: a matrix of another shape would be
    # read with the wrong row pitch, or transposed.
    T, H, Is = 3, 256, 640
    code = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)
    x, y, ws = torch.zeros((T, H), dtype=torch.float16), torch.zeros((T, H), dtype=torch.float16), torch.zeros(1 << 20)
    good = dict(wg=code(Is, H), sg=torch.zeros(5, 2), wu=code(Is, H), su=torch.zeros(5, 2), wd=code(H, Is),
                sd=torch.zeros(2, 5))
    call = lambda **kw: moe.moe_shared_forward_fp8(x, *{**good, **kw}.values(), y, ws)
    for kw in (dict(wd=code(Is, H)), dict(wg=code(Is, 2 * H)), dict(wu=code(Is, H + 64)), dict(wu=code(2 * Is, H)),
               dict(wu=code(Is - 64, H)), dict(wd=code(H, Is + 64)), dict(wd=code(2 * H, Is)),
               dict(sd=torch.zeros(5, 2)), dict(sg=torch.zeros(2, 5)), dict(su=torch.zeros(5, 3))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            call(**kw)
    for kw in ({}, dict(sg=torch.zeros(10), sd=torch.zeros(64)), dict(su=torch.zeros(6, 2))):
        with pytest.raises(TypeError, match="CUDA"):  # shapes and scales that are read as they are meant
            call(**kw)
