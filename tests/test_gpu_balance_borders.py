"""The balance loss on both sides of the borders between one block, one launch and two, and with several passes of one
block, against the oracle (needs a GB300). Tolerances: test_gpu_balance.py."""
import numpy as np
import pytest
import torch

from tests import test_gpu_balance as tb
from tests.balance_plan_shapes import BORDERS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score,half", [("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("T,E,k,S", sorted(BORDERS))
def test_border(T, E, k, S, score, half):
    l, ids, ragged = tb._inputs(T, E, k, S, half=half, masked=True)
    even = np.linspace(0, T, S + 1).astype(np.int32)  # no sequence is empty, where there are tokens enough
    cfg, b = tb.moe.moe_balance_config(score, 0.5), tb.Buffers(T, E, S)
    lg, ig = tb._cuda(l), tb._cuda(ids)
    for off in (even, ragged, even):
        o = tb._cuda(off)
        for t in (b.counts, b.tokens, b.mean, b.loss):
            t.fill_(-7)
        b.forward(cfg, lg, ig, o)
        c, n, L = tb._check_forward(b, l, ids, off, k, score, 0.5)
        d = torch.full((T, E), 3.0, device="cuda")
        tb.moe.moe_balance_loss_backward(cfg, lg, k, o, b.counts, b.tokens, None, d)
        tb._check_backward(d.double().cpu().numpy(), (0.0, 3.0), l, off, k, c, n, score, 0.5, 1.0, L)
