"""Scored router against the FP64 oracle (needs a GB300).

Ids are compared exactly, except for tokens whose order hinges on two computed
values closer than 1e-6 (FP32 scores and sums round at 6e-8 relative; either
order is right there): there the weights alone are compared. Weights: FP32
exponentials, one division and the renormalising sum, 1e-6 relative each at
most, so rtol 4e-6."""
import itertools

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as f8
from tests._lib import binding

pytestmark = pytest.mark.gpu

moe = binding() if torch.cuda.is_available() else None

MARGIN, RTOL = 1e-6, 4e-6


def _run(l, k, bias=None, stream=None, **cfg):
    dev = torch.device("cuda")
    T = l.shape[0]
    lt = l if isinstance(l, torch.Tensor) else torch.from_numpy(l).to(dev)
    ids = torch.full((T, k), -7, dtype=torch.int32, device=dev)
    w = torch.full((T, k), 7.0, dtype=torch.float32, device=dev)
    bad = torch.zeros(1, dtype=torch.int32, device=dev)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).to(dev)
    moe.moe_route_scored(moe.moe_route_config(**cfg), lt, k, b, ids, w, bad, stream)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy(), int(bad.item())


def _check(l, k, bias=None, **cfg):
    got = _run(l, k, bias, **cfg)
    ref = f8.route_scored(l, k, bias=bias, **cfg)
    clear = f8.closest_call(l, k, bias=bias, **cfg) > MARGIN
    assert clear.mean() > 0.9
    assert np.array_equal(got[0][clear], ref[0][clear])
    assert np.allclose(got[1], ref[1], rtol=RTOL, atol=1e-12)
    assert got[2] == ref[2]
    return got


def _bias(rng, E):
    return rng.permutation(np.linspace(-0.1, 0.1, E)).astype(np.float32)


@pytest.mark.parametrize("score,rank,biased,renorm", list(itertools.product(
    ["softmax", "sigmoid"], ["max", "top2"], [False, True], [False, True])))
@pytest.mark.parametrize("T,E,G,tg,k", [(1, 256, 8, 4, 8), (37, 60, 6, 3, 4), (5, 8, 8, 3, 3), (9, 96, 1, 1, 32),
                                        (3, 1024, 32, 5, 16)])
def test_matches_oracle(T, E, G, tg, k, score, rank, biased, renorm):
    rng = np.random.default_rng(E + T)
    l = (1.5 * rng.normal(size=(T, E))).astype(np.float32)
    _check(l, k, _bias(rng, E) if biased else None, score=score, n_groups=G, top_groups=tg, group_rank=rank,
           renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,G,k", [(1, 1, 1), (2, 2, 1), (33, 1, 7), (513, 1, 10), (1020, 17, 12), (1023, 31, 6),
                                   (999, 9, 9), (31, 31, 4)])
def test_odd_expert_counts(E, G, k):
    rng = np.random.default_rng(E)
    l = rng.normal(size=(11, E)).astype(np.float32)
    _check(l, k, _bias(rng, E), score="sigmoid", n_groups=G, top_groups=max(1, G // 2), group_rank="top2")


@pytest.mark.parametrize("T", [4099, 8192])
def test_many_tokens(T):
    rng = np.random.default_rng(T)
    l = rng.normal(size=(T, 64)).astype(np.float32)
    _check(l, 6, _bias(rng, 64), score="sigmoid", n_groups=4, top_groups=2, group_rank="top2", scale=1.5)


@pytest.mark.parametrize("T,E,G,tg,k,biased,rank", [(4096, 60, 6, 3, 4, False, "max"), (4097, 64, 1, 1, 16, True, "max"),
                                                     (5001, 48, 16, 5, 9, True, "top2"), (4100, 20, 1, 1, 7, False, "max")])
def test_many_tokens_few_experts(T, E, G, tg, k, biased, rank):
    # Half a warp per token; odd token counts, masked experts and tokens, a NaN and an infinity among them.
    rng = np.random.default_rng(T + E)
    l = rng.normal(size=(T, E)).astype(np.float32)
    l[rng.random(l.shape) < 0.4] = -np.inf
    l[5::97] = -np.inf
    l[7, 0], l[T - 1, E - 1], l[T // 2] = np.nan, np.inf, 0.25
    bias = _bias(rng, E) if biased else None
    cfg = dict(score="sigmoid", n_groups=G, top_groups=tg, group_rank=rank, scale=2.0)
    got = _run(l, k, bias, **cfg)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = f8.route_scored(l, k, bias=bias, **cfg)
        clear = f8.closest_call(l, k, bias=bias, **cfg) > MARGIN
    clear[T // 2] = True
    assert clear.mean() > 0.9 and np.array_equal(got[0][clear], ref[0][clear])
    assert np.allclose(got[1], ref[1], rtol=RTOL, atol=1e-12) and got[2] == ref[2]


def test_equals_moe_route_without_bias_and_groups():
    l = np.random.default_rng(5).normal(size=(300, 64)).astype(np.float32)
    l[:, 40:] = l[:, :24]  # exact ties
    dev = torch.device("cuda")
    for renorm in (False, True):
        ids = torch.empty((300, 8), dtype=torch.int32, device=dev)
        w = torch.empty((300, 8), dtype=torch.float32, device=dev)
        moe.moe_route(torch.from_numpy(l).to(dev), 8, renorm, ids, w)
        got = _run(l, 8, renorm=renorm)
        assert np.array_equal(got[0], ids.cpu().numpy())
        assert np.allclose(got[1], w.cpu().numpy(), rtol=RTOL)


def test_ties_go_to_the_lowest_index():
    l = np.zeros((3, 48), np.float32)
    l[1, ::2] = -0.0
    l[2, 40:] = 1.0
    for score in ("softmax", "sigmoid"):
        got = _run(l, 5, score=score, n_groups=6, top_groups=2, group_rank="top2")
        assert got[0].tolist() == [[0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [40, 41, 42, 43, 44]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("T", [64, 4100])
@pytest.mark.parametrize("score,renorm,units", [("sigmoid", False, 8), ("sigmoid", True, 20), ("softmax", False, 30)])
def test_weights_of_large_logits(score, renorm, units, T, dtype):
    # Logits of up to 80 either way, all representable in FP16 and their differences in FP32: what is left are the
    # roundings, in units of 2^-24 of the weight. Sigmoid: the exponential 2 (one ulp), the sum 1, the reciprocal
    # 2, the scale 1; renormalised: 5 each for the score and for the sum, 5 to add it up, the division and the
    # scale; softmax: the exponential 2, the normaliser's exponentials 4 + 1.44 |l - max| (of weight
    # exp(l - max) each: 14 on average at most), 8 to add them up, three products.
    rng = np.random.default_rng(T + units)
    c = np.linspace(-80, 78, T)[:, None] if score == "sigmoid" else 0.0
    l = c + (rng.uniform(0, 2, (T, 32)) if score == "sigmoid" else rng.uniform(-80, 80, (T, 32)))
    l = np.round(l * 16) / 16
    lt = torch.from_numpy(l.astype(np.float32)).to(dtype).cuda()
    got = _run(lt, 12, score=score, renorm=renorm, scale=1.5)
    ref = f8.route_scored(l, 12, score=score, renorm=renorm, scale=1.5)
    assert np.array_equal(got[0], ref[0])
    big = ref[1] > 2.0 ** -125
    assert big.mean() > 0.2
    assert (np.abs(got[1] - ref[1])[big] <= units * 2.0 ** -24 * ref[1][big]).all(), (
        np.abs(got[1] / ref[1] - 1)[big].max() * 2 ** 24)
    assert (got[1][~big] <= 2.0 ** -124).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [4000, 5000])
def test_close_values_keep_their_order(score, T):
    # Two experts whose score + bias are within a few FP32 roundings of each other: whichever
    # comes first does so for one pick and for two.
    rng = np.random.default_rng(T)
    for b in rng.uniform(0.02, 0.4, 40):
        if score == "softmax":  # s0 - s1 = tanh(d / 2) = b
            d = 2 * np.arctanh(b)
            base = rng.uniform(-2, 2, T)
        else:                   # s0 - s1 = b around s1 = base
            base = rng.uniform(-1, 0.2, T)
            s1 = 1 / (1 + np.exp(-base))
            d = -np.log(1 / (s1 + b) - 1) - base
        l = np.stack([base + d, base], 1).astype(np.float32)
        for _ in range(3):  # a few representable values to either side
            l[:, 0] = np.where(rng.random(T) < 0.5, np.nextafter(l[:, 0], np.float32(9)), np.nextafter(l[:, 0], np.float32(-9)))
        bias = [0.0, b]
        one, two = _run(l, 1, bias, score=score)[0], _run(l, 2, bias, score=score)[0]
        assert set(np.unique(one)) <= {0, 1} and (two.sum(1) == 1).all()
        assert np.array_equal(one[:, 0], two[:, 0]), int((one[:, 0] != two[:, 0]).sum())


def test_saturated_scores_are_ordered_by_logit():
    # 1 / (1 + exp(-40)) rounds to 1 in FP32: the logits still order the experts.
    l = (40.0 + np.random.default_rng(2).permutation(64)[None]).astype(np.float32)
    got = _run(l, 4, score="sigmoid")
    assert got[0].tolist() == [np.argsort(-l[0])[:4].tolist()] and np.allclose(got[1], 0.25)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G,rank", [(1, "max"), (4, "max"), (4, "top2")])
def test_masks_and_bad_tokens(score, biased, G, rank):
    rng = np.random.default_rng(7)
    l = rng.normal(size=(40, 32)).astype(np.float32)
    l[rng.random(l.shape) < 0.6] = -np.inf
    l[3] = -np.inf                      # none left
    l[4, 5], l[5, 31] = np.nan, np.inf
    l[6] = -np.inf
    l[6, 17] = 0.5                      # one left
    l[7] = np.finfo(np.float32).min     # the type's lowest value is a logit like any other
    l[8, 8:] = np.finfo(np.float32).min
    bias = _bias(rng, 32) if biased else None
    cfg = dict(score=score, n_groups=G, top_groups=max(1, G // 2), group_rank=rank)
    got = _run(l, 6, bias, **cfg)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = f8.route_scored(l, 6, bias=bias, **cfg)
        gap = f8.closest_call(l, 6, bias=bias, **cfg)
    clear = gap > MARGIN
    assert np.array_equal(got[0][clear], ref[0][clear]) and clear.sum() > 30
    assert np.allclose(got[1], ref[1], rtol=RTOL, atol=1e-12) and got[2] == ref[2] == 3
    assert got[0][6].tolist() == [17] + [-1] * 5


@pytest.mark.parametrize("T", [3, 4100])
def test_bias_of_the_lowest_value_ranks_above_no_expert(T):
    # Two experts biased by FP32's lowest value: their sum is still above that of a group without experts.
    l = np.zeros((T, 8), np.float32)
    l[:, :2] = l[:, 6:] = -np.inf
    bias = np.full(8, np.finfo(np.float32).min)
    cfg = dict(score="sigmoid", n_groups=4, top_groups=1, group_rank="top2")
    got = _run(l, 2, bias, **cfg)
    assert (got[0] == [2, 3]).all() and np.allclose(got[1], 0.5) and got[2] == 0
    assert f8.route_scored(l[:1], 2, bias=bias, **cfg)[0].tolist() == [[2, 3]]


def test_bias_masks_and_bad_bias():
    l = np.random.default_rng(8).normal(size=(9, 16)).astype(np.float32)
    bias = np.zeros(16, np.float32)
    bias[3:] = -np.inf
    got = _check(l, 5, bias, score="sigmoid")
    assert (got[0][:, 3:] == -1).all() and (got[0][:, :3] >= 0).all()
    for v in (np.nan, np.inf):
        bias[5] = v
        got = _run(l, 5, bias, score="sigmoid")
        assert (got[0] == -1).all() and not got[1].any() and got[2] == 9


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("E,pad", [(64, 0), (64, 64), (60, 5), (256, 1)])
def test_types_and_row_strides(dtype, E, pad):
    rng = np.random.default_rng(E + pad)
    full = torch.from_numpy(rng.normal(size=(50, E + pad)).astype(np.float32)).to(dtype).cuda()
    view = full[:, pad // 2:pad // 2 + E]
    bias = _bias(rng, E)
    cfg = dict(score="sigmoid", n_groups=4, top_groups=2, group_rank="top2", renorm=True, scale=2.5)
    got = _run(view, 6, bias, **cfg)
    l = view.float().cpu().numpy()
    ref = f8.route_scored(l, 6, bias=bias, **cfg)
    clear = f8.closest_call(l, 6, bias=bias, **cfg) > MARGIN
    assert np.array_equal(got[0][clear], ref[0][clear])
    assert np.allclose(got[1], ref[1], rtol=RTOL)


def test_rows_beyond_32_bit_offsets():
    # Row 40 starts 2.4e9 elements into the buffer (FP16, 4.8 GB).
    ld, T, E = 60_000_000, 41, 16
    buf = torch.zeros(ld * (T - 1) + E, dtype=torch.float16, device="cuda")
    view = torch.as_strided(buf, (T, E), (ld, 1))
    vals = np.random.default_rng(3).normal(size=(T, E)).astype(np.float16)
    view.copy_(torch.from_numpy(vals).cuda())
    got = _run(view, 4, score="sigmoid")
    ref = f8.route_scored(vals, 4, score="sigmoid")
    assert np.array_equal(got[0], ref[0]) and np.allclose(got[1], ref[1], rtol=RTOL)


def test_token_count_at_the_end_of_32_bits():
    # 2^31 - 1 tokens of one expert: the token number of the step after the last ones passes 2^31.
    T, dev, part = (1 << 31) - 1, torch.device("cuda"), 1 << 26
    l = torch.empty((T, 1), dtype=torch.float16, device=dev)
    for i in range(0, T, part):
        n = min(part, T - i)
        l[i:i + n, 0] = (torch.arange(i, i + n, device=dev) % 1009).float() / 128 - 4
    nan = torch.tensor([5, T // 2, T - 30000, T - 1], device=dev)
    l[nan] = float("nan")
    ids = torch.full((T, 1), -7, dtype=torch.int32, device=dev)
    w = torch.full((T, 1), 7.0, device=dev)
    bad = torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_route_scored(moe.moe_route_config(score="sigmoid", renorm=False), l, 1, None, ids, w, bad)
    assert int(bad) == 4 and (ids[nan] == -1).all() and not w[nan].any()
    ids[nan], w[nan], l[nan] = 0, 0.5, 0.0
    for i in range(0, T, part):
        assert not ids[i:i + part].any()
        ref = torch.sigmoid(l[i:i + part].double())
        assert ((w[i:i + part] - ref).abs() <= RTOL * ref).all()


def test_other_stream_and_repeatability():
    l = np.random.default_rng(4).normal(size=(500, 128)).astype(np.float32)
    lt = torch.from_numpy(l).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = _run(lt, 8, score="softmax", n_groups=8, top_groups=3, group_rank="top2")
    b = _run(lt, 8, stream=s, score="softmax", n_groups=8, top_groups=3, group_rank="top2")
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_refusals():
    dev = torch.device("cuda")
    l = torch.zeros((4, 16), device=dev)
    ids = torch.empty((4, 4), dtype=torch.int32, device=dev)
    w = torch.empty((4, 4), device=dev)
    for cfg, k in ((dict(n_groups=3), 2), (dict(n_groups=4, top_groups=5), 2), (dict(n_groups=8, top_groups=1), 3),
                   (dict(n_groups=0), 2), (dict(scale=float("nan")), 2), (dict(), 0), (dict(), 17)):
        with pytest.raises((moe.MoeError, ValueError)):
            moe.moe_route_scored(moe.moe_route_config(**cfg), l, k, None, ids, w)
    cfg = moe.moe_route_config()
    with pytest.raises(TypeError):
        moe.moe_route_scored(cfg, l.double(), 2, None, ids, w)
    with pytest.raises(ValueError):
        moe.moe_route_scored(cfg, l.t(), 2, None, ids, w)
    with pytest.raises(ValueError):
        moe.moe_route_scored(cfg, l, 8, None, ids, w)
    with pytest.raises(ValueError):
        moe.moe_route_scored(cfg, l, 4, torch.zeros(8, device=dev), ids, w)


def test_empty_batch():
    dev = torch.device("cuda")
    moe.moe_route_scored(moe.moe_route_config(), torch.empty((0, 16), device=dev), 4, None,
                         torch.empty((0, 4), dtype=torch.int32, device=dev), torch.empty((0, 4), device=dev))
    torch.cuda.synchronize()
