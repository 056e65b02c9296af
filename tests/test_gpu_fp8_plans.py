"""Every kernel instance that the FP8 product's plan can choose, against the
oracle (needs a GB300). Tolerances as in test_gpu_fp8.py."""
import numpy as np
import pytest
import torch

from tests.fp8_plan_shapes import GATE_UPS, PRODUCTS
from tests.test_gpu_fp8 import _check_ffn, _check_product, _ffn, _matmul, _quantize

pytestmark = pytest.mark.gpu


def _listed(table):
    return [pytest.param(*s, id="%d-%d_%dx%dx%d" % (*plan, *s)) for plan, sizes in table.items() for s in sizes]


def _acts(gen, rows, cols):
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x *= torch.where(torch.rand((cols,), generator=gen, device="cuda") < 0.01, 12.0, 1.0)
    return x.half().cpu().numpy()


def _weights(gen, rows, cols):
    # Each 128 x 128 block with a scale of its own, up to three times its neighbour's.
    s = torch.exp(torch.rand((-(-rows // 128), -(-cols // 128)), generator=gen, device="cuda"))
    s = s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return (0.02 * s * torch.randn((rows, cols), generator=gen, device="cuda")).half().cpu().numpy()


def _rows(T):
    """The edges of the token tiles and some between."""
    near = np.r_[0:3, 31:33, 127:130, 255:258, T // 2, T - 3:T, (T - 1) // 128 * 128]
    return np.unique(near[(near >= 0) & (near < T)])


@pytest.mark.parametrize("T,N,K", _listed(PRODUCTS))
def test_product_instances(T, N, K):
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    xq, xs = _quantize(_acts(gen, T, K), 1)
    wq, ws = _quantize(_weights(gen, N, K), 128)
    y = _matmul(xq, xs, wq, ws)
    assert not (y == 777.0).any()
    r = _rows(T)
    _check_product(y[r], xq[r], xs[r], wq, ws)


@pytest.mark.parametrize("T,Is,H", _listed(GATE_UPS))
def test_gate_up_instances(T, Is, H):
    gen = torch.Generator(device="cuda").manual_seed(T + Is + H)
    x = torch.randn((T, H), generator=gen, device="cuda").half().cpu().numpy()
    w = []
    for r, c in ((Is, H), (Is, H), (H, Is)):
        w += list(_quantize(_weights(gen, r, c), 128))
    y = _ffn(x, w)
    assert not (y == 777.0).any()
    r = _rows(T)
    _check_ffn(y[r], x[r], w)
