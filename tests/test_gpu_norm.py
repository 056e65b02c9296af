"""Norms before and after a block against the oracle (needs a GB300).

Tolerances. h is FP32 arithmetic on at most four factors and one sum: within
2^-21 of the sum of its terms' magnitudes M (with a post norm, whose own value
is off by 2^-19 of itself: 2^-18). y = (h - mean) r w: h's error and the mean's
(a sum of H values by threads and halving, 2^-19 of the mean magnitude) enter
times r |w|; r, from a sum of squares, is within 2^-19 of itself, and w + offset
and the products add 2^-22. An FP16 output adds half a step, 2^-11 of itself
(2^-25 among the subnormals), an FP32 one 2^-24. A code is within half a step,
2^-4, of the value over the scale (2^-10 scale among the subnormal codes)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from oracle import fp8_oracle as f8
from tests._lib import binding

pytestmark = pytest.mark.gpu

moe = binding() if torch.cuda.is_available() else None


def _cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _vec(rng, H, mean=1.0):
    return (mean + 0.3 * rng.normal(size=H)).astype(np.float16)


def _stream(rng, T, H, f32):
    x = rng.normal(size=(T, H)) * 1.5
    x[:, rng.random(H) < 0.02] *= 20
    return x.astype(np.float32 if f32 else np.float16)


def _half(v):
    return 2.0 ** -11 * np.abs(v) + 2.0 ** -25


def _y_bound(h, e_h, y, r, w, kind, b=None):
    """Error of y in FP32, from h's."""
    e_h = e_h + np.zeros(h.shape)
    y = np.abs(y) + (0.0 if b is None else np.abs(b.astype(np.float64)))  # the product before the bias at most
    if kind == "layer":
        e_h = e_h + 2.0 ** -19 * np.abs(h).mean(1, keepdims=True)
    # r's error from h's: relative 2 rms(e_h) r at most.
    e_r = 2.0 ** -19 + 2 * np.sqrt((e_h ** 2).mean(1, keepdims=True)) * r
    return r * np.abs(w) * e_h + (np.abs(y) + 1e-30) * (e_r + 2.0 ** -21) + 2.0 ** -22 * np.abs(y)


def _check_codes(q, s, y, e):
    """Codes and scales against y, off by e itself."""
    T, H = y.shape
    nb = f8.nblocks(H)
    for j in range(nb):
        c = slice(128 * j, min(128 * j + 128, H))
        m, em = np.abs(y[:, c]).max(1), e[:, c].max(1)
        assert (np.abs(s[:, j] - m / 448) <= em / 448 + 2.0 ** -22 * m / 448).all()
        got = q[:, c].astype(np.float64) * s[:, j:j + 1].astype(np.float64)
        # A code stands for y within half its step; the scale's own error moves all of them together.
        assert (np.abs(got - y[:, c]) <= 2.0 ** -4 * np.abs(y[:, c]) * 1.001 + s[:, j:j + 1] * 2.0 ** -10 + 2 * e[:, c]
                + np.abs(y[:, c]) * 2.0 ** -20).all()


SIZES = [(1, 8), (1, 2048), (3, 24), (5, 136), (7, 264), (9, 520), (2, 1032), (33, 2008), (4, 4096), (3, 4104), (2, 8192),
         (3, 8200), (2, 16384), (130, 64)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm(T, H, f32, kind):
    rng = np.random.default_rng(T * H)
    x, off = _stream(rng, T, H, f32), 1.0 if H % 24 == 0 else 0.0
    w, b = _vec(rng, H, 1 - off), _vec(rng, H, 0.0) if kind == "layer" else None
    y, r = bo.norm(x, w, b, kind, 1e-5, off)
    e = _y_bound(x.astype(np.float64), 0.0, y, r, w.astype(np.float64) + off, kind, b)
    cfg = moe.moe_norm_config(kind, 1e-5, off)
    out = torch.full((T, H), 7.0, dtype=torch.float16, device="cuda")
    fp8 = H % 16 == 0
    q = torch.zeros((T, H), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) if fp8 else None
    s = torch.full((T, f8.nblocks(H)), 9.0, device="cuda") if fp8 else None
    moe.moe_norm(cfg, _cuda(x), _cuda(w), _cuda(b), out, q, s)
    got = out.double().cpu().numpy()
    assert (np.abs(got - y) <= e + _half(y)).all(), np.abs(got - y).max()
    if fp8:
        _check_codes(q.float().cpu().numpy(), s.cpu().numpy(), y, e)
        q2, s2 = torch.zeros_like(q), torch.zeros_like(s)  # codes alone: the same ones
        moe.moe_norm(cfg, _cuda(x), _cuda(w), _cuda(b), None, q2, s2)
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "element"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("kind,f32", [("rms", False), ("rms", True), ("layer", False), ("layer", True)])
@pytest.mark.parametrize("T,H", [(1, 8), (1, 2048), (5, 264), (33, 2008), (2, 4112), (3, 8200), (2, 16384)])
def test_norm_residual(T, H, kind, f32, post, gate):
    rng = np.random.default_rng(T + H)
    br, res = (0.8 * rng.normal(size=(T, H))).astype(np.float16), _stream(rng, T, H, f32)
    w, pw = _vec(rng, H), _vec(rng, H)
    b, pb = (_vec(rng, H, 0.0), _vec(rng, H, 0.0)) if kind == "layer" else (None, None)
    g = {"none": None, "token": rng.normal(size=T).astype(np.float32), "channel": _vec(rng, H),
         "element": rng.normal(size=(T, H)).astype(np.float16)}[gate]
    sc, rs = 0.75, 1.25
    h, m = bo.residual(br, res, g, sc, rs, dict(w=pw, b=pb if post else None, kind=kind, eps=1e-6) if post else None)
    e_h = 2.0 ** -21 * m
    if post:  # the post norm's error, through the gate
        a, ra = bo.norm(br, pw, pb, kind, 1e-6)
        e_h = e_h + np.abs(sc * bo.gate_of(g, T, H)) * _y_bound(br.astype(np.float64), 0.0, a, ra, pw, kind, pb)
    y, r = bo.norm(h, w, b, kind, 1e-6)
    e_y = _y_bound(h, e_h, y, r, w, kind, b)
    dh = torch.full((T, H), 7.0, dtype=torch.float32 if f32 else torch.float16, device="cuda")
    dy = torch.full((T, H), 7.0, dtype=torch.float16, device="cuda")
    moe.moe_norm_residual(moe.moe_norm_config(kind, 1e-6), _cuda(br), _cuda(res), dh, _cuda(pw) if post else None,
                          _cuda(pb) if post else None, _cuda(g), sc, rs, _cuda(w), _cuda(b), dy)
    got = dh.double().cpu().numpy()
    assert (np.abs(got - h) <= e_h + (2.0 ** -24 * np.abs(h) if f32 else _half(h))).all(), np.abs(got - h).max()
    got = dy.double().cpu().numpy()
    assert (np.abs(got - y) <= e_y + _half(y)).all(), np.abs(got - y).max()


def _call(T, H, f32=False, seed=0):
    rng = np.random.default_rng(seed)
    return dict(branch=_cuda((0.8 * rng.normal(size=(T, H))).astype(np.float16)), residual=_cuda(_stream(rng, T, H, f32)),
                w=_cuda(_vec(rng, H)), post_w=_cuda(_vec(rng, H)))


def test_parts_of_the_residual_call():
    # h alone, y alone, no residual, codes: each as in the whole call.
    cfg, T, H = moe.moe_norm_config(), 37, 1040
    c = _call(T, H, True)
    new = lambda d=torch.float16: torch.empty((T, H), dtype=d, device="cuda")
    h, y, q, s = new(torch.float32), new(), new(torch.float8_e4m3fn), torch.empty((T, 9), device="cuda")
    moe.moe_norm_residual(cfg, c["branch"], c["residual"], h, w=c["w"], y=y, q=q, scales=s)
    h2, y2, q2, s2 = new(torch.float32), new(), new(torch.float8_e4m3fn), torch.empty((T, 9), device="cuda")
    moe.moe_norm_residual(cfg, c["branch"], c["residual"], h2)
    moe.moe_norm_residual(cfg, c["branch"], c["residual"], None, w=c["w"], y=y2)
    moe.moe_norm_residual(cfg, c["branch"], c["residual"], None, w=c["w"], q=q2, scales=s2)
    assert torch.equal(h, h2) and torch.equal(y, y2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s, s2)
    # y comes from h as moe_norm makes it from an FP32 h.
    moe.moe_norm(cfg, h, c["w"], None, y2, q2, s2)
    assert torch.equal(y, y2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    zero = torch.zeros((T, H), device="cuda")
    moe.moe_norm_residual(cfg, c["branch"], None, h2, scale=0.5)
    moe.moe_norm_residual(cfg, c["branch"], zero, h, scale=0.5)
    assert torch.equal(h, h2)


@pytest.mark.parametrize("f32", [False, True])
def test_in_place(f32):
    cfg, T, H = moe.moe_norm_config(), 65, 4112
    c = _call(T, H, f32)
    h, y = torch.empty_like(c["residual"]), torch.empty_like(c["branch"])
    moe.moe_norm_residual(cfg, c["branch"], c["residual"], h, c["post_w"], w=c["w"], y=y)
    r, br = c["residual"].clone(), c["branch"].clone()
    moe.moe_norm_residual(cfg, br, r, r, c["post_w"], w=c["w"], y=br)
    assert torch.equal(r, h) and torch.equal(br, y)
    if not f32:
        x = c["residual"].clone()
        moe.moe_norm(cfg, x, c["w"], None, x)
        moe.moe_norm(cfg, c["residual"], c["w"], None, y)
        assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_odd_values_stay_in_their_row(kind):
    cfg, T, H = moe.moe_norm_config(kind, 0.0), 6, 2064
    x = np.random.default_rng(5).normal(size=(T, H)).astype(np.float16)
    x[1, 100], x[2, 2063], x[3, 0], x[4] = np.nan, np.inf, -np.inf, 0.0
    x[5] = 6e-8  # the smallest subnormal: squares of 2^-48 still sum
    w = np.ones(H, np.float16)
    y = torch.empty((T, H), dtype=torch.float16, device="cuda")
    q, s = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((T, 17), device="cuda")
    moe.moe_norm(cfg, _cuda(x), _cuda(w), None, y, q, s)
    got, want = y.float().cpu().numpy(), bo.norm(x, w, None, kind, 0.0)[0]
    assert np.isnan(got[1]).all() and np.isnan(got[4]).all()  # NaN; 0 / 0
    assert np.isnan(got[2, 2063]) and np.isnan(got[3, 0])     # infinity times 0
    if kind == "rms":
        assert (got[2, :2063] == 0).all() and (got[3, 1:] == 0).all()
        assert np.allclose(got[5], 1.0, rtol=2.0 ** -10)
    assert np.allclose(got[0], want[0], rtol=2.0 ** -10, atol=2.0 ** -20)
    sc = s.cpu().numpy()
    assert np.isnan(sc[1]).all() and np.isnan(sc[2, 16]) and np.isnan(q.float().cpu().numpy()[1]).all()
    assert not np.isnan(sc[0]).any()
    if kind == "rms":
        assert (sc[2, :16] == 0).all()  # a block of zeros


def test_largest_values():
    cfg, H = moe.moe_norm_config(), 16384
    x = torch.full((2, H), 65504.0, dtype=torch.float16, device="cuda")
    w, y = torch.ones(H, dtype=torch.float16, device="cuda"), torch.empty((2, H), dtype=torch.float16, device="cuda")
    moe.moe_norm(cfg, x, w, None, y)
    assert torch.allclose(y.float(), torch.ones_like(y, dtype=torch.float32), rtol=2.0 ** -11)
    big = torch.full((1, H), 1e17, device="cuda")
    moe.moe_norm(cfg, big, w, None, y[:1])
    assert torch.allclose(y[:1].float(), torch.ones((1, H), device="cuda"), rtol=2.0 ** -11)


def test_beyond_32_bit_offsets():
    T, H = 300_000, 8192  # 2.46e9 elements
    cfg = moe.moe_norm_config()
    x = torch.empty((T, H), dtype=torch.float16, device="cuda").fill_(0.5)
    rows = [0, 1, 262_143, 262_144, 262_145, T - 1]
    rng = np.random.default_rng(2)
    part, w = _stream(rng, len(rows), H, False), _vec(rng, H)
    x[rows] = _cuda(part)
    y, q = torch.zeros_like(x), torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((T, 64), device="cuda")
    moe.moe_norm_residual(cfg, x, x, x, scale=0.0, w=_cuda(w), y=y, q=q, scales=s)
    want, r = bo.norm(part, w)
    got = y[rows].double().cpu().numpy()
    e = _y_bound(part.astype(np.float64), 2.0 ** -21 * np.abs(part.astype(np.float64)), want, r, w, "rms")
    assert (np.abs(got - want) <= e + _half(want)).all()
    _check_codes(q.view(torch.uint8)[rows].view(torch.float8_e4m3fn).float().cpu().numpy(), s[rows].cpu().numpy(), want, e)
    one = bo.norm(np.full((1, H), 0.5), w)[0]
    assert np.allclose(y[T - 7].double().cpu().numpy(), one[0], rtol=2.0 ** -10)


def test_many_short_rows():
    T, H = 1_000_003, 8
    x = torch.randn((T, H), device="cuda")
    w, y = torch.ones(H, dtype=torch.float16, device="cuda"), torch.zeros((T, H), dtype=torch.float16, device="cuda")
    moe.moe_norm(moe.moe_norm_config(), x, w, None, y)
    want = x.double() / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + 1e-6)
    assert ((y.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -18 * want.abs() + 2.0 ** -25).all()


def test_graph_and_stream():
    cfg, T, H = moe.moe_norm_config(), 19, 2048
    c = _call(T, H, True)
    h, y = torch.zeros((T, H), device="cuda"), torch.zeros((T, H), dtype=torch.float16, device="cuda")
    call = lambda: moe.moe_norm_residual(cfg, c["branch"], c["residual"], h, w=c["w"], y=y)
    call()
    want = h.clone(), y.clone()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        call()
    h.zero_(), y.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    c["branch"].mul_(0.5)  # replayed on new values
    graph.replay()
    call_h = h.clone()
    call()
    assert torch.equal(h, call_h) and not torch.equal(h, want[0])


def test_refusals():
    cfg, c = moe.moe_norm_config(), _call(4, 64)
    y = torch.empty((4, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="w"):
        moe.moe_norm(cfg, c["residual"], c["w"][:56], None, y)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_norm(cfg, c["residual"][:, ::2], c["w"], None, y)
    with pytest.raises(moe.MoeError):
        moe.moe_norm(cfg, c["residual"], c["w"], c["w"], y)  # an RMS norm has no bias
    with pytest.raises(moe.MoeError):
        moe.moe_norm(cfg, c["residual"], c["w"])
    with pytest.raises(moe.MoeError):
        moe.moe_norm_residual(cfg, c["branch"], c["residual"], None)
    with pytest.raises(moe.MoeError):
        moe.moe_norm_residual(cfg, c["branch"], c["residual"], None, y=y)
    with pytest.raises(TypeError):
        moe.moe_norm_residual(cfg, c["branch"], c["residual"], c["residual"].float())
    with pytest.raises(ValueError, match="gate"):
        moe.moe_norm_residual(cfg, c["branch"], c["residual"], y, gate=c["w"][:4])
    moe.moe_norm(cfg, c["residual"][:0], c["w"], None, y[:0])  # no tokens


@pytest.mark.parametrize("T,H", [(70_001, 64), (16_400, 264), (8300, 520), (8200, 776), (4200, 1032), (2101, 2008), (1100, 4104),
                                 (600, 8192), (300, 16384)])
@pytest.mark.parametrize("f32", [False, True])
def test_large_batches(T, H, f32):
    # Above 4 M elements the rows are shared otherwise: the same values as row by row in small batches.
    g = torch.Generator(device="cuda").manual_seed(T)
    br = torch.randn((T, H), generator=g, device="cuda").half()
    res = torch.randn((T, H), generator=g, device="cuda").to(torch.float32 if f32 else torch.float16)
    w, pw, gate = (torch.rand(H, generator=g, device="cuda").half() for _ in range(3))
    cfg = moe.moe_norm_config()
    for post in (None, pw):
        h, y = torch.full_like(res, 7.0), torch.full_like(br, 7.0)
        moe.moe_norm_residual(cfg, br, res, h, post, None, gate, 1.0, 1.0, w, None, y)
        a = br.double()
        if post is not None:
            a = a / torch.sqrt((a * a).mean(1, keepdim=True) + 1e-6) * pw.double()
        want = res.double() + gate.double() * a
        m = res.double().abs() + (gate.double() * a).abs()
        e = 2.0 ** -18 * m
        assert ((h.double() - want).abs() <= e + (2.0 ** -24 if f32 else 2.0 ** -11) * want.abs() + 2.0 ** -25).all()
        r = 1 / torch.sqrt((want * want).mean(1, keepdim=True) + 1e-6)
        n = want * r * w.double()
        e = r * w.double() * e + 2.0 ** -17 * n.abs()  # r's error from h's too
        assert ((y.double() - n).abs() <= e + 2.0 ** -11 * n.abs() + 2.0 ** -25).all()
    moe.moe_norm(cfg, res, w, None, y)
    want = res.double() / torch.sqrt((res.double() ** 2).mean(1, keepdim=True) + 1e-6) * w.double()
    assert ((y.double() - want).abs() <= (2.0 ** -11 + 2.0 ** -18) * want.abs() + 2.0 ** -25).all()
