"""Balance loss, per-expert counts and the gradient against the oracle (needs a GB300).

Counts and tokens are exact. A probability is a few FP32 operations and a sum
over E: within 2^-20 of itself (a logit of magnitude L adds 2^-23 L through its
difference from the largest). Means and the loss are sums of positive terms,
2^-18 relative with the order of their additions. A gradient is c p (f - dot),
off by 2^-19 of c p (f + dot), the magnitude its terms have."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from tests._lib import binding

pytestmark = pytest.mark.gpu

moe = binding() if torch.cuda.is_available() else None


def _cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _inputs(T, E, k, S, seed=0, half=False, masked=False, lo=0, hi=None):
    """Logits, ids with some holes, offsets (ragged, one sequence empty if S > 2) over tokens [lo, hi)."""
    rng = np.random.default_rng(seed + T * E + k)
    l = rng.normal(size=(T, E)) * 2 + rng.normal(size=E)
    if masked:
        l[rng.random((T, E)) < 0.4] = -np.inf
        l[::7] = -np.inf
    l = l.astype(np.float16 if half else np.float32)
    ids = np.argsort(-l.astype(np.float64) + 1e-9 * rng.random((T, E)), 1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < 0.05] = -1
    ids[rng.random((T, k)) < 0.02] = E + 3
    hi = T if hi is None else hi
    off = np.sort(rng.integers(lo, hi + 1, S + 1)).astype(np.int32)
    off[0], off[S] = lo, hi
    if S > 2:
        off[S // 2] = off[S // 2 - 1]
    return l, ids, off


class Buffers:
    def __init__(self, T, E, S):
        self.counts = torch.full((S, E), -5, dtype=torch.int32, device="cuda")
        self.tokens = torch.full((S,), -5, dtype=torch.int32, device="cuda")
        self.mean = torch.full((S, E), -5.0, device="cuda")
        self.loss = torch.full((1,), -5.0, device="cuda")
        self.work = torch.zeros(moe.moe_balance_workspace_bytes(T, E, S), dtype=torch.uint8, device="cuda")

    def forward(self, cfg, l, ids, off, stream=None):
        moe.moe_balance_loss(cfg, l, ids, off, self.counts, self.tokens, self.mean, self.loss, self.work, stream)


def _check_forward(b, l, ids, off, k, score, coef):
    c, n, mean, loss = bo.balance(l, ids, off, k, score, coef)
    assert np.array_equal(b.counts.cpu().numpy(), c) and np.array_equal(b.tokens.cpu().numpy(), n)
    L = np.abs(l[np.isfinite(l)].astype(np.float64)).max() if np.isfinite(l).any() else 0.0
    rel = 2.0 ** -18 + 2.0 ** -22 * L
    assert (np.abs(b.mean.cpu().numpy() - mean) <= rel * mean + 1e-38).all()
    assert abs(float(b.loss) - loss) <= rel * abs(loss) + 1e-38
    return c, n, L


def _check_backward(got, before, l, off, k, c, n, score, coef, grad, L):
    d, m, inside = bo.balance_grad(l, off, k, c, n, score, coef, grad)
    want = np.where(inside[:, None], before[0] + d, before[1])
    assert (np.abs(got - want) <= (2.0 ** -19 + 2.0 ** -22 * L) * m + 2.0 ** -24 * np.abs(want) + 1e-37).all()
    assert np.array_equal(got[~inside], np.broadcast_to(before[1], got.shape)[~inside])


SIZES = [(1, 1, 1, 1), (1, 256, 8, 1), (5, 4, 2, 1), (33, 8, 8, 3), (64, 60, 4, 2), (100, 64, 8, 1), (257, 65, 3, 9), (300, 100, 10, 4),
         (130, 128, 2, 2), (129, 130, 5, 5), (700, 256, 8, 16), (333, 257, 9, 3), (90, 511, 16, 2), (150, 512, 10, 7),
         (40, 516, 32, 3), (70, 1023, 4, 2), (200, 1024, 8, 5)]


@pytest.mark.parametrize("half,masked", [(False, False), (True, True), (False, True), (True, False)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S", SIZES)
def test_balance(T, E, k, S, score, half, masked):
    l, ids, off = _inputs(T, E, k, S, half=half, masked=masked)
    cfg, b = moe.moe_balance_config(score, 0.01), Buffers(T, E, S)
    lg, o = _cuda(l), _cuda(off)
    b.forward(cfg, lg, _cuda(ids), o)
    c, n, L = _check_forward(b, l, ids, off, k, score, 0.01)
    d = torch.full((T, E), 3.0, device="cuda")
    g = torch.full((1,), 1.5, device="cuda")
    moe.moe_balance_loss_backward(cfg, lg, k, o, b.counts, b.tokens, g, d)
    _check_backward(d.double().cpu().numpy(), (0.0, 3.0), l, off, k, c, n, score, 0.01, 1.5, L)


@pytest.mark.parametrize("E", [60, 64, 256, 300])
def test_one_sequence_without_offsets_and_optional_outputs(E):
    T, k = 500, 4
    l, ids, _ = _inputs(T, E, k, 1)
    cfg, b = moe.moe_balance_config("softmax", 1.0), Buffers(T, E, 1)
    b.forward(cfg, _cuda(l), _cuda(ids), None)
    c, n, L = _check_forward(b, l, ids, None, k, "softmax", 1.0)
    counts, tokens = torch.zeros_like(b.counts), torch.zeros_like(b.tokens)
    moe.moe_balance_loss(cfg, _cuda(l), _cuda(ids), None, counts, tokens, None, None, b.work)  # the counts alone
    assert torch.equal(counts, b.counts) and torch.equal(tokens, b.tokens)
    d, d2 = torch.empty((T, E), device="cuda"), torch.empty((T, E), device="cuda")
    moe.moe_balance_loss_backward(cfg, _cuda(l), k, None, counts, tokens, None, d)
    moe.moe_balance_loss_backward(cfg, _cuda(l), k, None, counts, tokens, torch.ones(1, device="cuda"), d2)
    assert torch.equal(d, d2)
    _check_backward(d.double().cpu().numpy(), (0.0, 0.0), l, None, k, c, n, "softmax", 1.0, 1.0, L)


@pytest.mark.parametrize("E,pad", [(60, 4), (60, 3), (256, 8), (255, 1)])
@pytest.mark.parametrize("half", [False, True])
def test_strides_padding_and_accumulation(E, pad, half):
    # Rows with a gap between them, tokens before the first and behind the last sequence, a gradient to add to.
    T, k, S = 401, 5, 6
    l, ids, off = _inputs(T, E, k, S, half=half, lo=17, hi=350)
    lg = torch.full((T, E + pad), float("nan"), dtype=torch.float16 if half else torch.float32, device="cuda")
    lg[:, :E] = _cuda(l)
    cfg, b = moe.moe_balance_config("sigmoid", 0.5), Buffers(T, E, S)
    b.forward(cfg, lg[:, :E], _cuda(ids), _cuda(off))
    c, n, L = _check_forward(b, l, ids, off, k, "sigmoid", 0.5)
    for acc, before in ((False, (0.0, 0.25)), (True, (0.25, 0.25))):
        d = torch.full((T, E + 2 * pad), 0.25, device="cuda")
        moe.moe_balance_loss_backward(cfg, lg[:, :E], k, _cuda(off), b.counts, b.tokens, None, d[:, :E], acc)
        _check_backward(d[:, :E].double().cpu().numpy(), before, l, off, k, c, n, "sigmoid", 0.5, 1.0, L)
        assert (d[:, E:] == 0.25).all()


def test_many_sequences():
    # A token each, most of a chunk's sequences empty, and more sequences than threads.
    for T, S, k in ((1, 65535, 1), (700, 1500, 2), (2000, 2000, 1)):
        E = 12
        rng = np.random.default_rng(S)
        l = rng.normal(size=(T, E)).astype(np.float32)
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        off = (np.arange(S + 1) if T == S else np.sort(rng.integers(0, T + 1, S + 1))).astype(np.int32)
        cfg, b = moe.moe_balance_config("softmax", 1.0), Buffers(T, E, S)
        b.forward(cfg, _cuda(l), _cuda(ids), _cuda(off))
        c, n, L = _check_forward(b, l, ids, off, k, "softmax", 1.0)
        d = torch.full((T, E), 9.0, device="cuda")
        moe.moe_balance_loss_backward(cfg, _cuda(l), k, _cuda(off), b.counts, b.tokens, None, d)
        _check_backward(d.double().cpu().numpy(), (0.0, 9.0), l, off, k, c, n, "softmax", 1.0, 1.0, L)


def test_nothing_left():
    # No tokens; only bad tokens; sequences without tokens.
    E, k = 16, 2
    cfg = moe.moe_balance_config("sigmoid", 1.0)
    b = Buffers(0, E, 3)
    b.forward(cfg, torch.empty((0, E), device="cuda"), torch.empty((0, k), dtype=torch.int32, device="cuda"),
              torch.zeros(4, dtype=torch.int32, device="cuda"))
    for t in (b.counts, b.tokens, b.mean, b.loss):
        assert (t == 0).all()
    l = np.full((5, E), -np.inf, np.float32)
    l[1, 3], l[2, 0] = np.nan, np.inf
    ids = np.full((5, k), -1, np.int32)
    off = np.array([0, 0, 5, 5], np.int32)
    b = Buffers(5, E, 3)
    b.forward(cfg, _cuda(l), _cuda(ids), _cuda(off))
    for t in (b.counts, b.tokens, b.mean, b.loss):
        assert (t == 0).all()
    d = torch.full((5, E), 9.0, device="cuda")
    moe.moe_balance_loss_backward(cfg, _cuda(l), k, _cuda(off), b.counts, b.tokens, None, d)
    assert (d == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(score):
    # Scores that are all saturated or all vanish, the type's lowest value as a mask.
    T, E, k = 8, 40, 3
    l = np.random.default_rng(1).normal(size=(T, E)).astype(np.float32)
    l[0] += 60
    l[1] -= 60
    l[2] -= 200
    l[3] *= 100
    l[4, 5:] = np.finfo(np.float32).min
    l[5, :39] = -np.inf
    l[6] = np.finfo(np.float32).min
    l[7, ::2] = -1000
    ids = np.argsort(-l, 1, kind="stable")[:, :k].astype(np.int32)
    cfg, b = moe.moe_balance_config(score, 1.0), Buffers(T, E, 1)
    b.forward(cfg, _cuda(l), _cuda(ids), None)
    p, good, rest = bo.probabilities(l, score)
    assert good.all()
    c, n, mean, loss = bo.balance(l, ids, None, k, score, 1.0)
    assert np.array_equal(b.counts.cpu().numpy(), c) and int(b.tokens) == T
    rel = 2.0 ** -18 + 2.0 ** -22 * 300  # logits up to 300 that are not masked
    assert (np.abs(b.mean.cpu().numpy() - mean) <= rel * mean + 1e-38).all()
    d = torch.empty((T, E), device="cuda")
    moe.moe_balance_loss_backward(cfg, _cuda(l), k, None, b.counts, b.tokens, None, d)
    want, m, _ = bo.balance_grad(l, None, k, c, n, score, 1.0)
    got = d.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= rel * m + 1e-37).all()


def test_gradient_against_differences():
    # The call's own losses: d loss is about 2^-20 of the loss, so the step is large and the bound counts its
    # curvature (third derivatives of a softmax are below 1).
    T, E, k = 12, 16, 2
    l, ids, off = _inputs(T, E, k, 2)
    cfg, b = moe.moe_balance_config("softmax", 1.0), Buffers(T, E, 2)
    o = _cuda(off)
    b.forward(cfg, _cuda(l), _cuda(ids), o)
    d = torch.empty((T, E), device="cuda")
    moe.moe_balance_loss_backward(cfg, _cuda(l), k, o, b.counts, b.tokens, None, d)
    got, step, c = d.cpu().numpy(), 0.03, b.counts.clone()
    f_max = float((c.float() * E / k / b.tokens[:, None].clamp(min=1)).max())
    for t, e in ((0, 0), (3, 5), (7, 15), (11, 2)):
        v = []
        for s in (step, -step):
            m = l.copy()
            m[t, e] += s
            b.forward(cfg, _cuda(m), _cuda(ids), o)
            v.append(float(b.loss))
        bound = f_max * step ** 2 / 6 + (abs(v[0]) + abs(v[1])) * 2.0 ** -22 / step
        assert abs((v[0] - v[1]) / (2 * step) - got[t, e]) <= bound


@pytest.mark.parametrize("T,E,k,S", [(257, 64, 8, 1), (5000, 256, 8, 7), (300, 1000, 4, 3)])
def test_same_bits_graphs_streams_and_a_shared_workspace(T, E, k, S):
    l, ids, off = _inputs(T, E, k, S)
    cfg, b = moe.moe_balance_config("softmax", 0.01), Buffers(T, E, S)
    lg, ig, o = _cuda(l), _cuda(ids), _cuda(off)
    d = torch.zeros((T, E), device="cuda")

    def step():
        b.forward(cfg, lg, ig, o)
        moe.moe_balance_loss_backward(cfg, lg, k, o, b.counts, b.tokens, b.loss, d)
    step()
    want = [t.clone() for t in (b.counts, b.tokens, b.mean, b.loss, d)]
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        step()
    for _ in range(5):
        for t in (b.counts, b.tokens, b.mean, b.loss, d):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((b.counts, b.tokens, b.mean, b.loss, d), want))
    # The workspace serves another, smaller batch, and is left as it has to be.
    b2 = Buffers(9, E, 1)
    b2.work = b.work
    b2.forward(cfg, lg[:9], ig[:9], None)
    step()
    assert all(torch.equal(x, y) for x, y in zip((b.counts, b.tokens, b.mean, b.loss, d), want))
    # Two streams at once, buffers and a workspace each.
    b3, st3 = Buffers(T, E, S), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        b.forward(cfg, lg, ig, o, st)
        b3.forward(cfg, lg, ig, o, st3)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((b.counts, b.tokens, b.mean, b.loss), want))
    assert all(torch.equal(x, y) for x, y in zip((b3.counts, b3.tokens, b3.mean, b3.loss), want))


def test_beyond_32_bit_offsets():
    T, E, k = (1 << 22) + 5, 1024, 1  # 4.3e9 logits
    l = torch.zeros((T, E), dtype=torch.float16, device="cuda")
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    ids[T - 3:] = 7
    l[T - 1] = float("-inf")
    off = torch.tensor([0, T - 4, T], dtype=torch.int32, device="cuda")
    cfg, b = moe.moe_balance_config("softmax", 1.0), Buffers(T, E, 2)
    b.forward(cfg, l, ids, off)
    assert b.tokens.tolist() == [T - 4, 3] and b.counts[0, 0] == T - 4
    assert b.counts[1, 0] == 1 and b.counts[1, 7] == 3
    assert torch.allclose(b.mean, torch.full_like(b.mean, 1 / E), rtol=2.0 ** -18)
    d = torch.full((T, E), 9.0, device="cuda")
    moe.moe_balance_loss_backward(cfg, l, k, off, b.counts, b.tokens, None, d)
    # p = 1/E, f = E c / n: d = (f - mean f) / (2 n E).
    f = E * b.counts[1].double() / 3
    want = (f - f.mean()) / (2 * 3 * E)
    assert torch.allclose(d[T - 2].double(), want, rtol=1e-4, atol=1e-9)
    assert (d[T - 1] == 0).all()
    f = E * b.counts[0].double() / (T - 4)
    want = (f - f.mean()) / (2 * (T - 4.0) * E)
    for t in (0, (1 << 21) + 3, T - 5):
        assert torch.allclose(d[t].double(), want, rtol=1e-4, atol=1e-14)


def test_decreasing_offsets_stay_in_bounds():
    # Their result is not defined; nothing outside the buffers changes.
    T, E, k, S = 300, 64, 2, 4
    l, ids, _ = _inputs(T, E, k, S)
    b = Buffers(T, E, S)
    off = torch.tensor([200, -5, 500, 100, 250], dtype=torch.int32, device="cuda")
    guard = torch.full((T + 2, E), 9.0, device="cuda")
    cfg = moe.moe_balance_config()
    b.forward(cfg, _cuda(l), _cuda(ids), off)
    moe.moe_balance_loss_backward(cfg, _cuda(l), k, off, b.counts, b.tokens, None, guard[1:T + 1])
    assert (guard[0] == 9.0).all() and (guard[T + 1] == 9.0).all()
    l, ids, off = _inputs(T, E, k, S)  # and the workspace serves on
    b.forward(cfg, _cuda(l), _cuda(ids), _cuda(off))
    _check_forward(b, l, ids, off, k, "softmax", 1.0)


def test_refusals():
    T, E, k = 8, 16, 2
    l, ids, off = _inputs(T, E, k, 1)
    b, cfg = Buffers(T, E, 1), moe.moe_balance_config()
    lg, ig = _cuda(l), _cuda(ids)
    with pytest.raises(ValueError):
        b.forward(cfg, lg, ig[:4], None)
    with pytest.raises(ValueError):
        b.forward(cfg, lg, ig, torch.zeros(3, dtype=torch.int32, device="cuda"))  # two sequences: counts too small
    with pytest.raises(TypeError):
        b.forward(cfg, lg.double(), ig, None)
    with pytest.raises(TypeError):
        b.forward(cfg, lg, ig.long(), None)
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(cfg, lg, ig, None, b.counts, b.tokens, b.mean, b.loss, b.work[:256])
    with pytest.raises(ValueError):
        moe.moe_balance_loss_backward(cfg, lg, k, None, b.counts, b.tokens, None, torch.zeros((T, E + 1), device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss_backward(cfg, lg, 17, None, b.counts, b.tokens, None, torch.zeros((T, E), device="cuda"))


@pytest.mark.parametrize("T,E,k,S", [(3000, 8, 2, 4), (9000, 64, 4, 40), (6000, 130, 4, 3), (20000, 256, 8, 1), (20000, 256, 2, 500),
                                     (3000, 300, 3, 2), (2500, 1000, 2, 6)])
def test_sequences_over_many_chunks_and_one_workspace_for_all(T, E, k, S):
    # Long sequences that many blocks share, short ones within a block; the workspace serves calls of other
    # sizes in between, whose layout differs.
    l, ids, off = _inputs(T, E, k, S)
    cfg, b = moe.moe_balance_config("sigmoid", 0.01), Buffers(20000, 1024, 500)
    other = Buffers(1, 1024, 500)
    other.work = b.work
    small = _inputs(300, 1024, 2, 500, seed=1)
    b.counts, b.tokens, b.mean = b.counts[:S, :E].contiguous(), b.tokens[:S], b.mean[:S, :E].contiguous()
    args = _cuda(l), _cuda(ids), _cuda(off)
    b.forward(cfg, *args)
    _check_forward(b, l, ids, off, k, "sigmoid", 0.01)
    want = [t.clone() for t in (b.counts, b.tokens, b.mean, b.loss)]
    other.forward(cfg, *[_cuda(v) for v in small])
    _check_forward(other, *small, 2, "sigmoid", 0.01)
    b.forward(cfg, *args)
    assert all(torch.equal(x, y) for x, y in zip((b.counts, b.tokens, b.mean, b.loss), want))


@pytest.mark.parametrize("T,E,k,S", [(5000, 1, 1, 2), (9001, 3, 2, 5), (4000, 5, 3, 1023), (4000, 64, 3, 1024), (3 * 128, 64, 2, 16),
                                     (3 * 128 + 1, 64, 2, 16), (384, 60, 2, 17), (96, 256, 4, 3), (97, 255, 4, 3), (24, 700, 2, 2),
                                     (25, 700, 2, 2), (41 * 32, 1000, 2, 3), (40 * 32, 1000, 2, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_borders_between_the_ways_of_joining(T, E, k, S, score):
    # One block, one launch, two; offsets in shared memory or not; fewest experts.
    l, ids, off = _inputs(T, E, k, S, masked=True)
    cfg, b = moe.moe_balance_config(score, 0.5), Buffers(T, E, S)
    lg, ig, o = _cuda(l), _cuda(ids), _cuda(off)
    for _ in range(2):  # the workspace is left as it has to be
        for t in (b.counts, b.tokens, b.mean, b.loss):
            t.fill_(-7)
        b.forward(cfg, lg, ig, o)
        c, n, L = _check_forward(b, l, ids, off, k, score, 0.5)
    d = torch.full((T, E), 3.0, device="cuda")
    moe.moe_balance_loss_backward(cfg, lg, k, o, b.counts, b.tokens, None, d)
    _check_backward(d.double().cpu().numpy(), (0.0, 3.0), l, off, k, c, n, score, 0.5, 1.0, L)


def test_runs_of_empty_sequences():
    # Hundreds of empty sequences at the front, between two tokens and at the end.
    T, E, k = 300, 20, 2
    l, ids, _ = _inputs(T, E, k, 1)
    off = np.concatenate([np.zeros(300), [40], np.full(700, 41), [150, 151], np.full(400, 299), np.full(200, 300)]).astype(np.int32)
    S = len(off) - 1
    cfg, b = moe.moe_balance_config("softmax", 1.0), Buffers(T, E, S)
    o = _cuda(off)
    b.forward(cfg, _cuda(l), _cuda(ids), o)
    c, n, L = _check_forward(b, l, ids, off, k, "softmax", 1.0)
    d = torch.full((T, E), 3.0, device="cuda")
    moe.moe_balance_loss_backward(cfg, _cuda(l), k, o, b.counts, b.tokens, None, d)
    _check_backward(d.double().cpu().numpy(), (0.0, 3.0), l, off, k, c, n, "softmax", 1.0, 1.0, L)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_long_sums_of_equal_probabilities(score):
    # 2^25 tokens of an untrained router: p = 1 / 60, whose rounding errors all have one sign.
    T, E, k = 1 << 25, 60, 1
    l = torch.zeros((T, E), dtype=torch.float16, device="cuda")
    ids = torch.arange(T, dtype=torch.int32, device="cuda").remainder_(E).view(T, 1)
    cfg, b = moe.moe_balance_config(score, 1.0), Buffers(T, E, 1)
    b.forward(cfg, l, ids, None)
    assert int(b.tokens) == T and int(b.counts.sum()) == T
    assert ((b.mean.double() * E - 1).abs() <= 2.0 ** -17).all()  # 2 sums of some 200 terms, and p's own 2^-20
    assert abs(float(b.loss) - 1) <= 2.0 ** -16
