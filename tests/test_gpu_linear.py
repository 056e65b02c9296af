"""The FP16 product with bias, activation and residual against the oracle (needs a GB300).

Tolerance, with A = sum |x w| + |bias|: the tensor cores round the running sum
every 16 terms, each time by at most 2^-23 of it. For terms of random sign the
running sum stays below 4 sqrt(K) of a term's size and A is about 0.64 K of it:
(K / 16) 2^-23 4 sqrt(K) / (0.64 K) A = 0.4 sqrt(K) 2^-23 A, 2^-18 A at K = 4096.
2^-18 A max(1, sqrt(K / 4096)) covers that and the joining of split sums. An
activation's slope is at most 1.13, its own FP32 error 2^-19 of |v| + 1; the
residual is one more FP32 sum, and the output one rounding."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from tests._lib import binding

pytestmark = pytest.mark.gpu

moe = binding() if torch.cuda.is_available() else None
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid"]


def _ops(T, N, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T + N + K)
    x = torch.randn((T, K), generator=g, device="cuda")
    w = torch.randn((N, K), generator=g, device="cuda") * (1.2 / K ** 0.5)
    return x.half(), w.half(), 0.5 * torch.randn(N, generator=g, device="cuda"), torch.randn((T, N), generator=g, device="cuda")


def _bound(v, A, act_v, y, K, f32, residual):
    """v: before the activation."""
    e = 2.0 ** -18 * max(1.0, (K / 4096) ** 0.5) * A
    e = 1.13 * e + 2.0 ** -19 * (np.abs(v) + 1) * (act_v is not v)
    if residual is not None:
        e = e + 2.0 ** -24 * (np.abs(act_v) + np.abs(residual))
    return e + (2.0 ** -24 * np.abs(y) if f32 else 2.0 ** -11 * np.abs(y) + 2.0 ** -25)


def _check(got, x, w, bias, act, res, f32):
    x, w = x.double().cpu().numpy(), w.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    r = None if res is None else res.double().cpu().numpy()
    v, A = bo.linear(x, w, b)
    av = bo.act(act, v) if act != "none" else v
    y = av if r is None else av + r
    e = _bound(v, A, av, y, x.shape[1], f32, r)
    d = np.abs(got.double().cpu().numpy() - y)
    assert (d <= e).all(), (d / e).max()


def _work(T, N, K):
    return torch.zeros(moe.moe_linear_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")


def _run(T, N, K, act="none", bias=True, residual=True, f32=False, seed=0):
    x, w, b, r = _ops(T, N, K, seed)
    typ = torch.float32 if f32 else torch.float16
    b, r = b if bias else None, r.to(typ) if residual else None
    y, ws = torch.full((T, N), 7.0, dtype=typ, device="cuda"), _work(T, N, K)
    moe.moe_linear(x, w, b, y, ws, act, r)
    _check(y, x, w, b, act, r, f32)
    assert moe.moe_workspace_flags(ws) == 0


SIZES = [(1, 1, 8), (1, 256, 2048), (1, 60, 2048), (2, 17, 24), (5, 1001, 72), (8, 16, 1000), (9, 130, 2064), (13, 2048, 4096),
         (16, 64, 512), (17, 1, 8), (17, 513, 2064), (33, 96, 520), (64, 2048, 1024), (77, 1001, 2064), (128, 256, 2048),
         (129, 129, 136), (200, 4096, 512), (256, 256, 4096), (300, 1004, 2056), (513, 2056, 264), (1000, 60, 2048),
         (1021, 777, 1032)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear(T, N, K, f32):
    _run(T, N, K, ACTS[(T + N + K) % 6], bias=(T + N) % 3 != 0, residual=(N + K) % 2 == 0, f32=f32)


@pytest.mark.parametrize("T,N,K", [(3, 40, 264), (16, 100, 2048), (100, 333, 264), (700, 520, 264)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("f32,bias,residual", [(False, True, True), (True, False, False), (True, True, True),
                                               (False, False, True), (False, True, False)])
def test_epilogues(T, N, K, act, f32, bias, residual):
    _run(T, N, K, act, bias, residual, f32, seed=1)


@pytest.mark.parametrize("T,N,K", [(2, 24, 65536), (40, 72, 65536), (300, 65536, 16), (7, 65536, 64)])
def test_limits(T, N, K):
    _run(T, N, K, "silu", True, True, True)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,N,K", [(1, 40, 136), (6, 40, 136), (50, 333, 264), (50, 336, 264), (600, 600, 264), (600, 601, 264)])
@pytest.mark.parametrize("pad", [8, 3])
def test_strided_rows(T, N, K, f32, pad):
    x, w, b, r = _ops(T, N, K)
    typ = torch.float32 if f32 else torch.float16
    X = torch.full((T, K + 24), float("nan"), dtype=torch.float16, device="cuda")
    X[:, :K] = x
    R, Y = torch.full((T, N + 2 * pad), 5.0, dtype=typ, device="cuda"), torch.full((T, N + pad), 7.0, dtype=typ, device="cuda")
    R[:, :N] = r.to(typ)
    ws = _work(T, N, K)
    moe.moe_linear(X[:, :K], w, b, Y[:, :N], ws, "gelu", R[:, :N])
    _check(Y[:, :N], x, w, b, "gelu", r.to(typ), f32)
    assert (Y[:, N:] == 7.0).all()  # between the rows: left as it was
    # The residual in place.
    moe.moe_linear(X[:, :K], w, b, R[:, :N], ws, "gelu", R[:, :N])
    assert torch.equal(R[:, :N], Y[:, :N]) and (R[:, N:] == 5.0).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [3, 40, 300])
def test_odd_values(T, act):
    # Saturated activations, NaN and infinities: each in its own rows and columns.
    N, K = 264, 72
    x, w, b, _ = _ops(T, N, K)
    b[0], b[1], b[2], b[3] = 1e4, -1e4, 200.0, -200.0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y = torch.empty((T, N), device="cuda")
    moe.moe_linear(x, w, b, y, _work(T, N, K), act)
    rows = [0] + list(range(3, T))
    _check(y[rows], x[rows], w, b, act, None, True)
    assert y[1].isnan().all()
    if act in ("none", "relu"):
        pos = w[:, 7] > 0
        assert (y[2][pos] == float("inf")).all()
        assert (y[2][w[:, 7] < 0] == (float("-inf") if act == "none" else 0.0)).all()
    if act == "sigmoid":
        assert (y[2] == (w[:, 7] > 0).float()).all()


def test_fp16_overflow_and_fp32_range():
    x = torch.full((20, 256), 255.0, dtype=torch.float16, device="cuda")
    w = torch.full((40, 256), 4.0, dtype=torch.float16, device="cuda")
    y16, y32 = torch.empty((20, 40), dtype=torch.float16, device="cuda"), torch.empty((20, 40), device="cuda")
    for T in (3, 20):
        moe.moe_linear(x[:T], w, None, y16[:T], _work(T, 40, 256))
        moe.moe_linear(x[:T], w, None, y32[:T], _work(T, 40, 256))
        assert (y16[:T] == float("inf")).all() and (y32[:T] == 261120.0).all()


def test_beyond_32_bit_offsets():
    T, N, K = 140_000, 16_000, 16  # 2.24e9 outputs
    x, w, b, _ = _ops(8, N, K)
    X = torch.zeros((T, K), dtype=torch.float16, device="cuda")
    rows = [0, 1, 134_216, 134_217, 134_218, 134_219, T - 2, T - 1]
    X[rows] = x
    Y = torch.full((T, N), 7.0, dtype=torch.float16, device="cuda")
    moe.moe_linear(X, w, b, Y, _work(T, N, K), "none", Y)
    r = torch.full((8, N), 7.0, dtype=torch.float16, device="cuda")
    _check(Y[rows], x, w, b, "none", r, False)
    assert torch.equal(Y[100_000], Y[2]) and torch.equal(Y[T - 3], Y[2])
    del X, Y
    # Few tokens of far rows.
    for T in (12, 40):
        X = torch.zeros((T, 300_000_000), dtype=torch.float16, device="cuda")
        x, w, b, _ = _ops(T, 72, 136)
        X[:, :136] = x
        Y = torch.zeros((T, 300_000_000), dtype=torch.float16, device="cuda")
        moe.moe_linear(X[:, :136], w, b, Y[:, :72], _work(T, 72, 136))
        _check(Y[:, :72], x, w, b, "none", None, False)
        del X, Y


@pytest.mark.parametrize("T,N,K", [(4, 256, 2048), (60, 512, 2048), (600, 1024, 512)])
def test_same_bits_in_batches_graphs_and_streams(T, N, K):
    x, w, b, r = _ops(T, N, K)
    y, ws = torch.empty((T, N), dtype=torch.float16, device="cuda"), _work(T, N, K)
    call = lambda: moe.moe_linear(x, w, b, y, ws, "silu", r16)
    r16 = r.half()
    call()
    want = y.clone()
    for _ in range(5):
        y.zero_()
        call()
        assert torch.equal(y, want)
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        call()
        call()
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    # Two streams at once, a workspace each.
    y2, ws2, st2 = torch.empty_like(y), _work(T, N, K), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        moe.moe_linear(x, w, b, y, ws, "silu", r16, st)
        moe.moe_linear(x, w, b, y2, ws2, "silu", r16, st2)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(y2, want)


def test_workspace_serves_smaller_batches():
    N, K = 520, 264
    ws = _work(700, N, K)
    for T in (700, 1, 16, 17, 129, 300, 5):
        x, w, b, _ = _ops(T, N, K)
        y = torch.empty((T, N), device="cuda")
        moe.moe_linear(x, w, b, y, ws)
        _check(y, x, w, b, "none", None, True)


def test_refusals():
    x, w, b, r = _ops(4, 16, 64)
    y, ws = torch.empty((4, 16), device="cuda"), _work(4, 16, 64)
    for kw in (dict(bias=b[:8]), dict(y=y[:, :8]), dict(residual=r[:3]), dict(y=y.t()), dict(residual=r.t().contiguous().t())):
        a = dict(x=x, w=w, bias=b, y=y, workspace=ws, residual=None)
        with pytest.raises(ValueError):
            moe.moe_linear(**{**a, **kw})
    for kw in (dict(x=x.float()), dict(w=w.float()), dict(bias=b.half()), dict(y=y.double()), dict(residual=r.half())):
        a = dict(x=x, w=w, bias=b, y=y, workspace=ws, residual=None)
        with pytest.raises(TypeError):
            moe.moe_linear(**{**a, **kw})
    with pytest.raises(moe.MoeError):
        moe.moe_linear(x, w, b, y, ws[:0])
    with pytest.raises(moe.MoeError):  # rows that do not start on 16 bytes
        moe.moe_linear(torch.zeros((4, 68), dtype=torch.float16, device="cuda")[:, :64], w, b, y, ws)
    with pytest.raises(KeyError):
        moe.moe_linear(x, w, b, y, ws, "tanh")
    moe.moe_linear(x[:0], w, b, y[:0], ws)


@pytest.mark.parametrize("T,N,K", [(8, 2500, 520), (11, 2432, 4104), (16, 100, 6000), (10, 2433, 4096), (9, 7290, 136), (16, 7301, 80)])
def test_every_variant_of_the_weight_stream(T, N, K):
    _run(T, N, K, "none", True, True, True)
    _run(T, N, K, "silu", False, False, False, seed=3)


def test_all_kernels_at_once():
    """Each kernel on a stream of its own, all running together: the bits of a call alone."""
    shapes = [(4, 256, 2048), (16, 2048, 4096), (60, 512, 2048), (64, 2048, 2048), (600, 1024, 512), (2048, 2048, 512)]
    runs = []
    for T, N, K in shapes:
        x, w, b, _ = _ops(T, N, K)
        for dt in (torch.float16, torch.float32):
            y, ws = torch.empty((T, N), dtype=dt, device="cuda"), _work(T, N, K)
            moe.moe_linear(x, w, b, y, ws, "silu")
            runs.append((x, w, b, y, ws, y.clone(), torch.cuda.Stream()))
            y.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, b, y, ws, _, st in runs:
            moe.moe_linear(x, w, b, y, ws, "silu", None, st)
    torch.cuda.synchronize()
    for _, _, _, y, ws, want, _ in runs:
        assert torch.equal(y, want) and moe.moe_workspace_flags(ws) == 0
