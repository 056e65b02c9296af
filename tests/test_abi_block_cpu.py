"""Host-side argument checks of the norms, the FP16 product and the balance loss (no GPU)."""
import ctypes

import pytest
import torch

from tests._lib import binding

moe = binding()
lib = moe._lib


def test_norm_arguments():
    ok = moe.moe_norm_config()
    n = lambda cfg=ok, typ=0, T=0, H=64, b=None, q=None: lib.moe_norm(cfg, None, typ, T, H, None, b, None, q, None, None)
    assert n() == moe.MOE_OK
    assert n(T=1) == moe.MOE_ERR_ARG and "NULL" in moe.moe_last_error()
    for kw in (dict(cfg=None), dict(typ=2), dict(T=-1), dict(H=0), dict(H=12), dict(H=16392), dict(H=24, q=16),
               dict(b=16)):
        assert n(**kw) == moe.MOE_ERR_ARG, kw
    assert n(H=16384) == n(cfg=moe.moe_norm_config("layer"), b=16) == moe.MOE_OK
    for c in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(weight_offset=float("nan"))):
        assert n(cfg=moe.moe_norm_config(**c)) == moe.MOE_ERR_ARG, c
    bad = moe.moe_norm_config()
    bad.kind = 2
    assert n(cfg=bad) == moe.MOE_ERR_ARG
    with pytest.raises(KeyError):
        moe.moe_norm_config("group")
    assert ctypes.sizeof(ok) == 12
    P = 4096  # never read: the checks end the call before any launch
    full = lambda x=P, w=P, y=P, q=None, s=None: lib.moe_norm(ok, x, 1, 1, 64, w, None, y, q, s, None)
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(q=P), dict(s=P), dict(x=P + 8), dict(w=P + 2),
               dict(y=P + 4), dict(q=P + 8, s=P), dict(q=P, s=P + 2)):
        assert full(**kw) == moe.MOE_ERR_ARG, kw


def test_norm_residual_arguments():
    ok, P = moe.moe_norm_config("layer"), 4096

    def f(cfg=ok, branch=P, res=P, typ=1, T=1, H=64, pw=None, pb=None, gate=None, kind=0, scale=1.0, rscale=1.0, h=P,
          w=None, b=None, y=None, q=None, s=None):
        return lib.moe_norm_residual(cfg, branch, res, typ, T, H, pw, pb, gate, kind, scale, rscale, h, w, b, y, q, s,
                                     None)
    assert f(T=0) == moe.MOE_OK
    for kw in (dict(cfg=None), dict(branch=None), dict(typ=3), dict(H=20), dict(kind=4), dict(kind=-1), dict(kind=1),
               dict(scale=float("inf")), dict(rscale=float("nan")), dict(h=None), dict(y=P), dict(q=P, w=P),
               dict(s=P, w=P, y=P), dict(pb=P), dict(branch=P + 8), dict(res=P + 8), dict(h=P + 8),
               dict(kind=1, gate=P + 2), dict(kind=2, gate=P + 8), dict(kind=3, gate=P + 8), dict(pw=P + 2),
               dict(w=P, y=P + 2), dict(H=24, w=P, q=P, s=P), dict(cfg=moe.moe_norm_config(), b=P),
               dict(cfg=moe.moe_norm_config(), pw=P, pb=P)):
        assert f(**kw) == moe.MOE_ERR_ARG, kw


def test_linear_arguments():
    P = 4096

    def f(x=P, ldx=None, T=1, K=64, w=P, N=8, bias=None, act=0, r=None, ldr=8, y=P, typ=1, ldy=None, ws=P, nb=1 << 20):
        return lib.moe_linear(x, K if ldx is None else ldx, T, K, w, N, bias, act, r, ldr, y, typ,
                              N if ldy is None else ldy, ws, nb, None)
    assert f(T=0) == moe.MOE_OK
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ws=None), dict(K=4), dict(K=0), dict(K=65544), dict(N=0),
               dict(N=65537), dict(T=-1), dict(T=(1 << 20) + 1), dict(ldx=56), dict(ldx=68), dict(ldy=7),
               dict(r=P, ldr=7), dict(ldx=1 << 31), dict(ldy=1 << 31), dict(r=P, ldr=1 << 31), dict(act=6),
               dict(act=-1), dict(typ=2), dict(x=P + 8), dict(w=P + 8), dict(y=P + 8), dict(r=P + 4), dict(bias=P + 2),
               dict(ws=P + 16)):
        assert f(**kw) == moe.MOE_ERR_ARG, kw
    assert f(nb=0) == moe.MOE_ERR_CAPACITY
    assert moe.moe_linear_workspace_bytes(1, 8, 12) == 0 and moe.moe_linear_workspace_bytes(-1, 8, 16) == 0
    for N, K in ((1, 8), (256, 2048), (65536, 8), (4096, 65536)):
        sizes = [moe.moe_linear_workspace_bytes(T, N, K) for T in (0, 1, 2, 8, 9, 16, 17, 64, 128, 1000, 1 << 20)]
        assert sizes == sorted(sizes) and sizes[0] >= 256


def test_balance_arguments():
    ok, P = moe.moe_balance_config(), 4096

    def f(cfg=ok, l=P, typ=0, ld=16, T=4, E=16, ids=P, k=2, off=None, S=1, counts=P, tokens=P, mean=P, loss=P, ws=P,
          nb=1 << 30):
        return lib.moe_balance_loss(cfg, l, typ, ld, T, E, ids, k, off, S, counts, tokens, mean, loss, ws, nb, None)
    bad = [dict(cfg=None), dict(T=-1), dict(T=(1 << 27) + 1), dict(E=0, k=1), dict(E=1025, ld=2000), dict(k=0), dict(k=17),
           dict(k=33, E=64, ld=64), dict(T=1 << 27, k=16), dict(S=0, off=P), dict(S=65536, off=P), dict(S=2),
           dict(typ=2), dict(ld=15), dict(l=None), dict(l=P + 2), dict(off=P + 2)]
    for kw in bad + [dict(ids=None), dict(counts=None), dict(tokens=None), dict(ws=None), dict(ids=P + 2),
                     dict(counts=P + 1), dict(tokens=P + 2), dict(mean=P + 2), dict(loss=P + 2), dict(ws=P + 64)]:
        assert f(**kw) == moe.MOE_ERR_ARG, kw
    assert f(nb=256) == moe.MOE_ERR_CAPACITY
    for c in (dict(coef=float("inf")), dict(coef=float("nan"))):
        assert f(cfg=moe.moe_balance_config(**c)) == moe.MOE_ERR_ARG
    odd = moe.moe_balance_config()
    odd.score = 2
    assert f(cfg=odd) == moe.MOE_ERR_ARG

    def b(cfg=ok, l=P, typ=0, ld=16, T=4, E=16, k=2, off=None, S=1, counts=P, tokens=P, g=None, d=P, ldd=16):
        return lib.moe_balance_loss_backward(cfg, l, typ, ld, T, E, k, off, S, counts, tokens, g, d, ldd, 0, None)
    assert b(T=0, l=None) == moe.MOE_OK
    for kw in bad + [dict(counts=None), dict(tokens=None), dict(d=None), dict(ldd=15), dict(d=P + 2), dict(g=P + 2)]:
        assert b(**kw) == moe.MOE_ERR_ARG, kw
    assert moe.moe_balance_workspace_bytes(-1, 8, 1) == moe.moe_balance_workspace_bytes(1, 1025, 1) == 0
    assert moe.moe_balance_workspace_bytes(1, 8, 0) == moe.moe_balance_workspace_bytes(1, 8, 65536) == 0
    sizes = [moe.moe_balance_workspace_bytes(T, 256, 7) for T in (0, 1, 31, 32, 33, 500, 5000, 1 << 20, 1 << 27)]
    assert sizes == sorted(sizes)


def test_shapes_in_the_binding():
    # Checked before any pointer is taken, so tensors of the host do.
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    f = lambda *s: torch.zeros(s)
    cfg = moe.moe_norm_config()
    with pytest.raises(TypeError, match="float32 or float16"):
        moe.moe_norm(cfg, torch.zeros(2, 64, dtype=torch.bfloat16), h(64), None, h(2, 64))
    with pytest.raises(ValueError, match="residual"):
        moe.moe_norm_residual(cfg, h(2, 64), h(2, 72), None)
    with pytest.raises(ValueError, match="h must"):
        moe.moe_norm_residual(cfg, h(2, 64), h(2, 64), h(3, 64))
    for g in (f(64), h(2), f(3), f(2, 64), h(64, 2)):
        with pytest.raises(ValueError, match="gate"):
            moe._gate(g, 2, 64)
    with pytest.raises(ValueError, match="columns"):
        moe.moe_linear(h(2, 64), h(8, 72), None, h(2, 8), None)
    with pytest.raises(KeyError):
        moe._ACTS["tanh"]
    for t, kw in ((h(2, 64), {}), (torch.zeros(1), {})):
        with pytest.raises(TypeError, match="CUDA"):
            moe._rows(t, "x", (2, 64), (torch.float16,))
    with pytest.raises(TypeError, match="CUDA"):
        moe.moe_balance_loss(moe.moe_balance_config(), f(2, 8), None, None, None, None, None, None, None)


def test_block_arguments():
    P = 4096

    def block(**kw):
        f = dict(shape=moe.moe_expert_shape(256, 128, 64), experts=16, top_k=4, n_slots=16, shared_inter=0,
                 norm=moe.moe_norm_config(), route=moe.moe_route_config(), scale=1.0, residual_scale=1.0, norm_w=P, norm_b=None,
                 gate_w=P, gate_b=None, route_bias=None, pool=P, slot_of=P, shared_g=None, shared_u=None, shared_d=None,
                 post_w=None, post_b=None)
        return moe.moe_block(*{**f, **kw}.values())

    def f(b=None, h=P, typ=0, T=2, ids=P, w=P, lg=None, ws=P, nb=1 << 30, **kw):
        return lib.moe_block_forward(block(**kw) if b is None else b, h, typ, T, ids, w, lg, ws, nb, None)
    assert f(T=0) == moe.MOE_OK
    assert lib.moe_block_forward(None, P, 0, 0, P, P, None, P, 0, None) == moe.MOE_ERR_ARG
    layer, S = moe.moe_norm_config("layer"), dict(shared_inter=128, shared_g=P, shared_u=P, shared_d=P)
    assert f(T=0, norm=layer, norm_b=P, post_w=P, post_b=P, **S) == moe.MOE_OK
    assert f(T=0, shape=moe.moe_expert_shape(100, 128, 64)) == moe.MOE_ERR_SHAPE
    for kw in (dict(T=-1), dict(T=16385), dict(typ=2), dict(experts=0), dict(top_k=0), dict(top_k=17), dict(n_slots=0),
               dict(shared_inter=100, shared_g=P, shared_u=P, shared_d=P), dict(shared_inter=-64), dict(shared_g=P),
               {**S, "shared_d": None}, dict(norm_w=None), dict(gate_w=None), dict(pool=None), dict(slot_of=None),
               dict(norm_b=P), dict(post_b=P), dict(norm=layer, post_b=P), dict(scale=float("nan")),
               dict(residual_scale=float("inf")), dict(norm=moe.moe_norm_config(eps=-1.0)),
               dict(route=moe.moe_route_config(n_groups=3)), dict(norm_w=P + 8), dict(gate_w=P + 2), dict(pool=P + 16),
               dict(slot_of=P + 2), dict(gate_b=P + 2), dict(route_bias=P + 1), {**S, "shared_u": P + 8},
               dict(h=None), dict(ids=None), dict(w=None), dict(ws=None), dict(h=P + 8), dict(lg=P + 4), dict(ids=P + 2),
               dict(ws=P + 64)):
        assert f(**kw) == moe.MOE_ERR_ARG, kw
    assert f(nb=4096) == moe.MOE_ERR_CAPACITY
    b = block(**S)
    assert moe.moe_block_workspace_bytes(b, -1) == 0
    assert moe.moe_block_workspace_bytes(block(shape=moe.moe_expert_shape(100, 128, 64)), 4) == 0
    assert moe.moe_block_workspace_bytes(b, 4) > moe.moe_block_workspace_bytes(block(), 4) > 4 * (256 * 4 + 16 * 4)


def test_block_checks_the_experts_path_before_any_launch():
    # Small batches whose picks' intermediates exceed a block's shared memory on the GEMV path. Without a GPU a
    # launch would end in MOE_ERR_CUDA.
    P, none = 4096, None
    for inter, k in ((4096, 32), (8192, 16)):
        b = moe.moe_block(moe.moe_expert_shape(64, inter, 64), 64, k, 64, 0, moe.moe_norm_config(), moe.moe_route_config(),
                          1.0, 1.0, P, none, P, none, none, P, P, none, none, none, none, none)
        for T in (1, 2, 8):
            assert lib.moe_block_forward(b, P, 0, T, P, P, none, P, 1 << 40, none) == moe.MOE_ERR_UNSUPPORTED, (inter, k, T)
            assert "GEMV path" in moe.moe_last_error()


def test_balance_workspace_of_more_tokens_than_a_call_takes():
    most = 1 << 27
    assert moe.moe_balance_workspace_bytes(most, 1024, 65535) > 0
    for T in (most + 1, 1 << 30, (1 << 31) - 32, (1 << 31) - 1):
        assert moe.moe_balance_workspace_bytes(T, 256, 4) == 0, T


def test_block_workspace_of_arguments_that_a_call_refuses():
    def size(T, k=8, experts=64, Is=0):
        b = moe.moe_block(moe.moe_expert_shape(256, 128, 64), experts, k, 64, Is)
        return moe.moe_block_workspace_bytes(b, T)
    assert 0 < size(1) < size(8192) and size(2048, 32, 1024, 65536) > 0
    for a in ((8193,), (1 << 28,), ((1 << 31) - 1,), (2049, 32), (1, 33), (1, 8, 1025), (1, 8, (1 << 31) - 1), (1, 8, 64, 65600)):
        assert size(*a) == 0, a
