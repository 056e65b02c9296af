"""Pins of the FP8 and scored-routing oracle: hand values, closed forms and
the special cases it reduces to (CPU)."""
import numpy as np
import torch

from oracle import fp8_oracle as f8
from oracle import moe_oracle


def test_code_values_match_the_type():
    mine = f8.code_values()
    theirs = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(mine), np.isnan(theirs)) and np.isnan(mine).sum() == 2
    assert np.array_equal(mine[~np.isnan(mine)], theirs[~np.isnan(mine)])
    assert mine[0x7E] == 448.0 and mine[1] == 2.0 ** -9


def test_encode_rounds_to_nearest_even():
    # Between 1 (0x38) and 1.125 (0x39): the midpoint goes to the even code.
    assert f8.encode(np.array([1.0, 1.0625, 1.0626, 1.125, 1.1875])).tolist() == [0x38, 0x38, 0x39, 0x39, 0x3A]
    assert f8.encode(np.array([-1e9, 448.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [0xFE, 0x7E, 0x00, 0x02]
    v = np.random.default_rng(0).normal(size=20000).astype(np.float32) * 40
    theirs = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f8.encode(v), theirs)


def test_quantize_hand_block():
    x = np.zeros((2, 256), np.float16)
    x[0, 0], x[0, 1], x[0, 130] = 2.0, -1.0, 0.5
    q, s = f8.quantize(x, 1)
    assert s.tolist() == [[np.float32(2) / np.float32(448), np.float32(0.5) / np.float32(448)], [0, 0]]
    assert f8.decode(q[0, [0, 1, 130]]).tolist() == [448.0, -224.0, 448.0] and not q[1].any()
    q, s = f8.quantize(x, 128)
    assert s.shape == (1, 2)


def test_widen_matmul_closed_form():
    # Codes 1.0 everywhere: y = sum over blocks of (columns in block) * xs * ws.
    T, N, K = 3, 130, 160
    xq, wq = np.full((T, K), 0x38, np.uint8), np.full((N, K), 0x38, np.uint8)
    xs = np.array([[1.0, 2.0], [0.5, 1.0], [3.0, 0.0]])
    ws = np.array([[2.0, 4.0], [1.0, 8.0]])
    y = f8.matmul(xq, xs, wq, ws)
    want = 128 * xs[:, :1] * ws[None, :, 0] + 32 * xs[:, 1:] * ws[None, :, 1]
    assert np.allclose(y[:, [0, 129]], want)


def test_route_scored_reduces_to_route():
    l = np.random.default_rng(1).normal(size=(40, 60)).astype(np.float32)
    for renorm in (True, False):
        ids, w, bad = f8.route_scored(l, 5, renorm=renorm)
        rid, rw = moe_oracle.route(l, 5, renorm)[:2]
        assert bad == 0 and np.array_equal(ids, rid) and np.allclose(w, rw, rtol=1e-12)


def test_route_scored_hand_case():
    # Groups {0,1}, {2,3}, {4,5}; sigmoid(0) = 1/2. The bias lifts expert 5, not its weight.
    l = np.zeros((1, 6), np.float32)
    bias = [0.0, 0.1, 0.0, 0.05, 0.0, 0.3]
    ids, w, _ = f8.route_scored(l, 2, "sigmoid", 3, 2, "max", True, 2.0, bias)
    assert ids.tolist() == [[5, 1]] and np.allclose(w, [[1.0, 1.0]])
    ids, _, _ = f8.route_scored(l, 3, "sigmoid", 3, 1, "max", False, 1.0, bias)
    assert ids.tolist() == [[5, 4, -1]]
    # One large and one small against two middling: the sum of two ranks otherwise than the largest.
    l = np.array([[3.0, -9.0, 1.0, 1.0]], np.float32)
    assert f8.route_scored(l, 1, "sigmoid", 2, 1, "max", True, 1.0)[0].tolist() == [[0]]
    assert f8.route_scored(l, 1, "sigmoid", 2, 1, "top2", True, 1.0)[0].tolist() == [[2]]


def test_route_scored_masks():
    ninf = -np.inf
    l = np.array([[ninf, 1, ninf, 0], [ninf] * 4, [np.nan, 0, 0, 0], [0, np.inf, 0, 0]], np.float32)
    ids, w, bad = f8.route_scored(l, 3, "softmax", renorm=True)
    assert ids.tolist() == [[1, 3, -1], [-1] * 3, [-1] * 3, [-1] * 3] and bad == 3
    assert w[0, 2] == 0 and abs(w[0].sum() - 1) < 1e-12 and not w[1:].any()
