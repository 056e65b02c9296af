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
