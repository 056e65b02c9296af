"""Errors of moe_linear's long sums (needs a GB300).

Terms of one sign are the worst case of an accumulator that cuts its running
sum off: all cuts go one way. Products here lie in [1/4, 1). The bounds count a
cut per 16 terms of at most one unit in the last place, 2^-23 of the running
sum, which over an accumulator's n cuts adds up to (n + 1) / 2 2^-23 of its
result if the terms are equal; 1.1 covers their spread.
FP32 results: accumulators of 512 terms, n = 32, then FP32 sums of K / 512 of
them (the weight stream: of K / 512 steps of 64 per warp), each rounded by 2^-24
of a running sum that is half the result on average; 8 more sums join warps,
segments or ranks.
FP16 results above 16 tokens: n = 512 (8192 terms), 16 sums of them and of ranks;
then one rounding, half a unit in FP16's last place.
Measured, a cut is 1.7 units on average (3.5 2^-24 of the running sum), not less
than one: the addends are cut off too where they are aligned. The accumulators
are short enough for the bounds all the same."""
import numpy as np
import pytest
import torch

from tests import test_gpu_linear as tl
from tests.linear_accuracy_shapes import LONG, SEGMENTED, STREAM

pytestmark = pytest.mark.gpu

moe = tl.moe


def _e32(K):
    return 1.1 * 33 / 2 * 2.0 ** -23 + (K / 1024 + 8) * 2.0 ** -24


E16 = 1.1 * 513 / 2 * 2.0 ** -23 + 16 * 2.0 ** -24


def _one_sign(T, N, K, f32):
    """y, exact."""
    g = torch.Generator(device="cuda").manual_seed(T + N + K)
    x, w = ((0.5 + 0.5 * torch.rand(s, generator=g, device="cuda")).clamp(max=0.9995).half() for s in ((T, K), (N, K)))
    y, ws = torch.empty((T, N), dtype=torch.float32 if f32 else torch.float16, device="cuda"), tl._work(T, N, K)
    moe.moe_linear(x, w, None, y, ws)
    xd = x.double()
    exact = torch.cat([xd @ part.double().t() for part in w.split(1024)], 1)
    assert moe.moe_workspace_flags(ws) == 0
    return y.double(), exact


def _check(T, N, K, f32):
    y, exact = _one_sign(T, N, K, f32)
    rel = ((y - exact).abs() / exact).max().item()
    if f32:
        assert rel <= _e32(K), (T, N, K, rel / 2.0 ** -24)
    else:
        half = torch.exp2(torch.floor(torch.log2(exact)) - 11)
        e = _e32(K) if T <= 16 else E16
        over = (((y - exact).abs() - half) / exact).max().item()
        assert over <= e, (T, N, K, over / 2.0 ** -24)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("plan", sorted(LONG), ids=lambda p: f"{p[0]}x{p[1]}")
def test_terms_of_one_sign(plan, f32):
    assert torch.cuda.get_device_properties(0).multi_processor_count == 152  # the plans are listed for
    for T, N, K in LONG[plan]:
        _check(T, N, K, f32)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,N,K", STREAM)
def test_terms_of_one_sign_in_the_weight_stream(T, N, K, f32):
    _check(T, N, K, f32)


@pytest.mark.parametrize("T,N", [(1, 256), (8, 64), (16, 256), (64, 256), (1000, 60), (8192, 256)])
def test_router_logits(T, N):
    # Terms of random sign, K = 2048. A cut goes towards zero by 0.36 2^-23 of the running sum on average (half a unit,
    # a unit 0.72 of 2^-23 of a value), which after i of an accumulator's n cuts is sqrt(i / n) of its result: 2 n / 3
    # times 0.36 2^-23 in all, for n = 32 7.7 2^-23 = 0.9e-6 (one accumulator for all of K, n = 128: 31 2^-23 = 3.7e-6).
    K = 2048
    g = torch.Generator(device="cuda").manual_seed(T + N)
    x = torch.randn((T, K), generator=g, device="cuda").half()
    w = (torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).half()
    y = torch.empty((T, N), device="cuda")
    moe.moe_linear(x, w, None, y, tl._work(T, N, K))
    exact = x.double() @ w.double().t()
    rms = lambda v: float(np.sqrt(float((v * v).mean())))
    assert rms(y.double() - exact) <= 1.5e-6 * rms(exact), rms(y.double() - exact) / rms(exact)


@pytest.mark.parametrize("plan", sorted(LONG), ids=lambda p: f"{p[0]}x{p[1]}")
def test_long_sums_through_the_epilogue(plan):
    # FP16 results that are added up from segments, with bias, activation and residual.
    tl._run(*LONG[plan][0], "silu", True, True, False)


@pytest.mark.parametrize("plan", sorted(SEGMENTED), ids=lambda p: f"{p[0]}x{p[1]}")
@pytest.mark.parametrize("pad,rpad", [(8, 8), (3, 8), (8, 3), (1, 5), (4, 4)])
def test_strides_of_segmented_pairs(plan, pad, rpad):
    for T, N, K in SEGMENTED[plan]:
        x, w, b, r = tl._ops(T, N, K)
        R = torch.full((T, N + rpad), 5.0, dtype=torch.float16, device="cuda")
        Y = torch.full((T, N + pad), 7.0, dtype=torch.float16, device="cuda")
        R[:, :N] = r.half()
        ws = tl._work(T, N, K)
        moe.moe_linear(x, w, b, Y[:, :N], ws, "gelu", R[:, :N])
        tl._check(Y[:, :N], x, w, b, "gelu", r.half(), False)
        assert (Y[:, N:] == 7.0).all() and (R[:, N:] == 5.0).all()
        moe.moe_linear(x, w, b, R[:, :N], ws, "gelu", R[:, :N])  # in place
        assert torch.equal(R[:, :N], Y[:, :N]) and (R[:, N:] == 5.0).all()
        assert moe.moe_workspace_flags(ws) == 0
