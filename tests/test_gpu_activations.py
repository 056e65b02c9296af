"""moe_linear's activations at every FP16 value up to 14 (needs a GB300): x W^T has one term, so v is exact.

Bounds relative to the result, in units of 2^-24 (half a unit in FP32's last
place), s the sigmoid's own value:
  sigmoid, silu  expf 2 units in the last place (4), the sum 1, the division 2
                 units (4): 9. FP16 results above 16 tokens: 2^v of the special-
                 function unit 2^-22 (4), its exponent 1.5 |v| (1 - s), the sum 1,
                 1/v 2, a product 1.
  gelu_tanh      u = c (v + 0.044715 v^3), every factor and sum rounded: 6.5 of
                 itself, so 6.5 |2 u| (1 - s) in s, and the sigmoid's own.
  gelu           Phi by erfc: 4 units (8), its argument 1.5 of itself, v^2 times
                 that in the tail; products 3. (By e^(-v^2/2): the exponent is
                 rounded to 1.5 v^2 too.)
Then one rounding, half a step of the output's type. A sigmoid below 2^-126 may
count as 0."""
import math

import pytest
import torch

from tests import test_gpu_linear as tl

pytestmark = pytest.mark.gpu

moe = tl.moe


def _exact(act, v):
    if act == "relu":
        return v.clamp(min=0.0), torch.zeros_like(v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5)), 1.5 * v * v + 11
    u2 = 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3) if act == "gelu_tanh" else v
    s, rest = torch.sigmoid(u2), torch.sigmoid(-u2)
    exponent = u2.abs() * rest
    return s * (1.0 if act == "sigmoid" else v), 9 + 1.5 * exponent + (6.5 * exponent if act == "gelu_tanh" else 0.0)


def _half_step(y, f32):
    if f32:
        return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -126))) - 24)
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -14))) - 11)


def _values():
    h = torch.arange(0x4B01, dtype=torch.int16, device="cuda").view(torch.float16)  # 0 to 14
    return torch.cat([h, -h])


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T", [1, 12, 40, 600])
def test_every_value(T, f32, act):
    # The values in W, T equal tokens of one column.
    v = _values()
    N = v.numel()
    w = torch.zeros((N, 8), dtype=torch.float16, device="cuda")
    w[:, 0] = v
    x = torch.zeros((T, 8), dtype=torch.float16, device="cuda")
    x[:, 0] = 1.0
    y, ws = torch.full((T, N), 7.0, dtype=torch.float32 if f32 else torch.float16, device="cuda"), tl._work(T, N, 8)
    moe.moe_linear(x, w, None, y, ws, act)
    want, units = _exact(act, v.double())
    bound = units * 2.0 ** -24 * want.abs() + _half_step(want, f32) + 14 * 2.0 ** -126
    err = (y.double() - want).abs() / bound
    worst = int(err.max(0)[0].argmax())
    assert (err <= 1.0).all(), (float(v[worst]), float(want[worst]), float(y[0, worst]), float(err.max()))
