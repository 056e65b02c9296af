"""Every kernel instance that moe_linear can choose, at sizes that reach it, FP16 and FP32 results, with and
without residual (needs a GB300)."""
import pytest
import torch

from tests import test_gpu_linear as tl
from tests.linear_plan_shapes import PRODUCTS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("plan", sorted(PRODUCTS), ids=lambda p: f"{p[0]}x{p[1]}")
@pytest.mark.parametrize("f32", [False, True])
def test_instance(plan, f32):
    assert torch.cuda.get_device_properties(0).multi_processor_count == 152  # the plans are listed for
    for i, (T, N, K) in enumerate(PRODUCTS[plan]):
        for residual in (False, True):
            tl._run(T, N, K, tl.ACTS[(i + residual) % 5 if T * N < 1 << 22 else 2 * residual], residual != f32, residual, f32,
                    seed=i)


# Rows of y and the residual at pitches that TMA can and cannot address, N that ends inside 16 bytes.
STRIDED = {(-256, 1): [(303, 6448, 1016), (302, 4932, 1016), (306, 4961, 984)],
           (-128, 1): [(432, 1160, 264), (314, 348, 104), (297, 345, 88)]}


@pytest.mark.parametrize("plan", sorted(STRIDED), ids=lambda p: f"{p[0]}x{p[1]}")
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("pad,rpad", [(8, 8), (3, 8), (8, 3), (1, 5), (4, 4)])
def test_strides_of_the_pair_kernels(plan, f32, pad, rpad):
    for T, N, K in STRIDED[plan]:
        x, w, b, r = tl._ops(T, N, K)
        typ = torch.float32 if f32 else torch.float16
        R = torch.full((T, N + rpad), 5.0, dtype=typ, device="cuda")
        Y = torch.full((T, N + pad), 7.0, dtype=typ, device="cuda")
        R[:, :N] = r.to(typ)
        ws = tl._work(T, N, K)
        tl.moe.moe_linear(x, w, b, Y[:, :N], ws, "silu", R[:, :N])
        tl._check(Y[:, :N], x, w, b, "silu", r.to(typ), f32)
        assert (Y[:, N:] == 7.0).all() and (R[:, N:] == 5.0).all()
        tl.moe.moe_linear(x, w, b, R[:, :N], ws, "silu", R[:, :N])  # in place
        assert torch.equal(R[:, :N], Y[:, :N]) and (R[:, N:] == 5.0).all()
