"""FP8 quantisation, block-scaled product and shared FFN against the oracle
(needs a GB300).

Quantisation is compared bit for bit (each step is one FP32 operation).
Product: y is one rounding to FP16 (2^-11 relative, 2^-25 absolute among the
subnormals) of sums held in FP32; with A = sum |terms|, 2^-20 A covers the
order and the alignment of a few thousand FP32 additions of a block and the
joining of the blocks. FFN: the same, plus one code step for every element of
h that lies so near a rounding boundary that h's own error can move it."""
import numpy as np
import pytest
import torch

from int4_routed_expert_moe_gb300 import synth
from oracle import fp8_oracle as f8
from oracle import moe_oracle
from tests._lib import binding
from tests.gpu_util import LayerPool

pytestmark = pytest.mark.gpu

moe = binding() if torch.cuda.is_available() else None


def _acts(rng, T, K):
    x = rng.normal(size=(T, K))
    x[:, rng.random(K) < 0.01] *= 12
    return x.astype(np.float16)


def _weights(rng, N, K):
    return (rng.normal(size=(N, K)) * 0.02 * np.exp(0.3 * rng.normal(size=(N, 1)))).astype(np.float16)


def _codes(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().view(torch.float8_e4m3fn)


def _quantize(x, br, stream=None):
    R, C = x.shape
    xt = torch.from_numpy(x).cuda()
    q = torch.zeros((R, C), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((-(-R // br), f8.nblocks(C)), 9.0, device="cuda")
    torch.cuda.synchronize()
    moe.moe_quantize_fp8(xt, q, s, br, stream)
    torch.cuda.synchronize()
    return q.view(torch.uint8).cpu().numpy(), s.cpu().numpy()


# ---- quantisation -----------------------------------------------------------
@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("R,C", [(1, 16), (1, 2048), (7, 144), (128, 128), (129, 272), (300, 1040), (33, 8192)])
def test_quantize_bit_exact(R, C, br):
    x = _acts(np.random.default_rng(R * C), R, C)
    x[R // 2, :128] = 0
    q, s = f8.quantize(x, br)
    gq, gs = _quantize(x, br)
    assert np.array_equal(gs, s) and np.array_equal(f8.decode(gq), f8.decode(q))


@pytest.mark.parametrize("br", [1, 128])
def test_quantize_extremes(br):
    x = np.zeros((260, 400), np.float16)
    x[0, :] = 6e-8                 # the smallest subnormal
    x[1, 0], x[1, 1] = 65504, 6e-8
    x[131, 200] = -65504
    x[140, 390] = 2.0 ** -14
    q, s = f8.quantize(x, br)
    gq, gs = _quantize(x, br)
    assert np.array_equal(gs, s) and np.array_equal(f8.decode(gq), f8.decode(q))


@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("v", [np.nan, np.inf, -np.inf])
def test_quantize_nonfinite_block(v, br):
    x = _acts(np.random.default_rng(1), 200, 304)
    x[130, 130] = v
    q, s = f8.quantize(x, br)
    gq, gs = _quantize(x, br)
    assert np.array_equal(np.isnan(gs), np.isnan(s)) and np.isnan(gs).sum() == 1
    assert np.array_equal(np.nan_to_num(gs), np.nan_to_num(s))
    a, b = f8.decode(gq), f8.decode(q)
    assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.nan_to_num(a), np.nan_to_num(b))


@pytest.mark.parametrize("br", [1, 128])
def test_quantize_codes_equal_eager(br):
    # The codes of x * (448.0 / amax) in PyTorch, ties between two codes included:
    # amax with few significant bits makes many of them.
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((1024, 2048), generator=g, device="cuda").half()
    x[:512] = (x[:512] * 32).round().clamp(-96, 96) / 32
    x[::128, ::128] = torch.tensor([3.0, 3.5, 7.0, 5.25], device="cuda").half().repeat(4)
    b = x.float().view(1024 // br, br, 16, 128)
    want = (b * (448.0 / b.abs().amax((1, 3), keepdim=True))).to(torch.float8_e4m3fn).view(1024, 2048)
    q = torch.empty_like(want)
    s = torch.empty((1024 // br, 16), device="cuda")
    moe.moe_quantize_fp8(x, q, s, br)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


def test_quantize_beyond_32_bit_offsets():
    R, C = 300_000, 8192  # 2.46e9 elements
    x = torch.empty((R, C), dtype=torch.float16, device="cuda").fill_(0.5)
    rows = [0, 1, 262_143, 262_144, 262_145, R - 1]
    part = _acts(np.random.default_rng(2), len(rows), C)
    x[rows] = torch.from_numpy(part).cuda()
    q = torch.empty((R, C), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.empty((R, C // 128), device="cuda")
    moe.moe_quantize_fp8(x, q, s, 1)
    gq, gs = q.view(torch.uint8)[rows].cpu().numpy(), s[rows].cpu().numpy()
    rq, rs = f8.quantize(part, 1)
    assert np.array_equal(gs, rs) and np.array_equal(f8.decode(gq), f8.decode(rq))
    assert (s[5] == 0.5 / 448).all() and (q[R - 7].float() == 448).all()


def test_quantize_more_than_2_29_blocks():
    # 2^29 + 1000 rows of one block each (16 columns): block numbers times eight lanes pass 32 bits.
    R, C = (1 << 29) + 1000, 16
    x = torch.full((R, C), 0.5, dtype=torch.float16, device="cuda")
    rows = [0, 1, 999, 1000, (1 << 28) + 3, (1 << 29) - 1, 1 << 29, (1 << 29) + 1, (1 << 29) + 500, R - 1]
    part = _acts(np.random.default_rng(4), len(rows), C)
    x[rows] = torch.from_numpy(part).cuda()
    q = torch.zeros((R, C), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((R, 1), 9.0, device="cuda")
    moe.moe_quantize_fp8(x, q, s, 1)
    rq, rs = f8.quantize(part, 1)
    assert np.array_equal(s[rows].cpu().numpy(), rs)
    assert np.array_equal(f8.decode(q.view(torch.uint8)[rows].cpu().numpy()), f8.decode(rq))
    assert int((s == 0.5 / 448).sum()) >= R - len(rows)  # every other row holds halves
    assert (q.view(torch.uint8)[R - 1000:R - 600:7] == 0x7E).float().mean() > 0.9


def test_quantize_other_stream():
    x = _acts(np.random.default_rng(3), 100, 512)
    a, b = _quantize(x, 1), _quantize(x, 1, torch.cuda.Stream())
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_quantize_refusals():
    def call(x, q, s, br):
        moe.moe_quantize_fp8(x, q, s, br)
    z = lambda r, c, d=torch.float16: torch.zeros((r, c), dtype=torch.float32, device="cuda").to(d)
    f = torch.float8_e4m3fn
    with pytest.raises(moe.MoeError):
        call(z(4, 40), z(4, 40, f), torch.zeros(4, device="cuda"), 1)
    with pytest.raises(moe.MoeError):
        call(z(4, 64), z(4, 64, f), torch.zeros(4, device="cuda"), 2)
    with pytest.raises(moe.MoeError):  # misaligned codes
        call(z(1, 64), z(1, 80, f).reshape(-1)[1:65].reshape(1, 64), torch.zeros(1, device="cuda"), 1)
    with pytest.raises(ValueError):
        call(z(4, 256), z(4, 256, f), torch.zeros(7, device="cuda"), 1)
    with pytest.raises(TypeError):
        call(z(4, 64, torch.float32), z(4, 64, f), torch.zeros(4, device="cuda"), 1)
    call(z(0, 64), z(0, 64, f), torch.zeros(0, device="cuda"), 1)


# ---- product ------------------------------------------------------------------
def _matmul(xq, xs, wq, ws, stream=None):
    T, K = xq.shape
    N = wq.shape[0]
    args = [_codes(xq), torch.from_numpy(xs).cuda(), _codes(wq), torch.from_numpy(ws).cuda()]
    y = torch.full((T, N), 777.0, dtype=torch.float16, device="cuda")
    ws_ = torch.zeros(moe.moe_matmul_fp8_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    moe.moe_matmul_fp8(*args, y, ws_, stream)
    torch.cuda.synchronize()
    assert moe.moe_workspace_flags(ws_) == 0
    return y.cpu().numpy()


def _check_product(y, xq, xs, wq, ws):
    xv, wv = f8.widen(xq, xs, 1), f8.widen(wq, ws, 128)
    ref, A = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -20 * A + 2.0 ** -25
    err = np.abs(y.astype(np.float64) - ref)
    assert (err <= tol).all(), (err / tol).max()


SHAPES = [(1, 1, 16), (1, 128, 128), (1, 4096, 2048), (2, 1000, 144), (3, 129, 272), (8, 127, 4096), (16, 640, 2064),
          (17, 65, 80), (33, 257, 1024), (64, 512, 640), (65, 96, 2048), (77, 1001, 2064), (127, 256, 256),
          (128, 128, 8192), (129, 300, 512), (200, 2048, 208), (256, 256, 384), (257, 513, 1040), (512, 4096, 128),
          (1030, 72, 2064), (1500, 1500, 512)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_product_matches_oracle(T, N, K):
    rng = np.random.default_rng(T * N + K)
    xq, xs = f8.quantize(_acts(rng, T, K), 1)
    wq, ws = f8.quantize(_weights(rng, N, K), 128)
    _check_product(_matmul(xq, xs, wq, ws), xq, xs, wq, ws)


def test_product_large_sampled():
    rng = np.random.default_rng(9)
    T, N, K = 2500, 4096, 1024
    x, w = _acts(rng, T, K), _weights(rng, N, K)
    xq, xs = _quantize(x, 1)
    wq, ws = _quantize(w, 128)
    y = _matmul(xq, xs, wq, ws)
    r = [0, 1, 127, 128, 129, 255, 256, 1000, 2047, 2304, 2431, 2432, 2499]
    _check_product(y[r], xq[r], xs[r], wq, ws)


@pytest.mark.parametrize("T,N,K", [(2048, 1001, 1040), (2048, 1004, 528), (1900, 1288, 272), (600, 4096, 272)])
def test_product_many_tokens_sampled(T, N, K):
    # Many-token tiles with ragged edges: rows that TMA can store and rows that it cannot (N odd, N even).
    rng = np.random.default_rng(T + N)
    xq, xs = _quantize(_acts(rng, T, K), 1)
    wq, ws = _quantize(_weights(rng, N, K), 128)
    y = _matmul(xq, xs, wq, ws)
    r = np.unique(np.r_[0:4, 30:34, 126:130, 254:258, T // 2, T - 140:T - 120, T - 3:T])
    _check_product(y[r], xq[r], xs[r], wq, ws)
    assert not (y == 777.0).any()


def test_product_scales_of_every_block():
    # Codes 1.0 throughout, scales distinct powers of two per block: each block's sum is exact,
    # so every misplaced scale shows.
    T, N, K = 140, 300, 400
    xq, wq = np.full((T, K), 0x38, np.uint8), np.full((N, K), 0x38, np.uint8)
    rng = np.random.default_rng(0)
    xs = (2.0 ** rng.integers(-6, 0, (T, 4))).astype(np.float32)
    ws = (2.0 ** rng.integers(-6, 0, (3, 4))).astype(np.float32)
    _check_product(_matmul(xq, xs, wq, ws), xq, xs, wq, ws)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_product_zero_and_nan_blocks(T):
    rng = np.random.default_rng(T)
    x = _acts(rng, T, 512)
    x[0, 128:256] = 0
    x[T - 1, 300] = np.inf
    xq, xs = f8.quantize(x, 1)
    wq, ws = f8.quantize(_weights(rng, 200, 512), 128)
    y = _matmul(xq, xs, wq, ws)
    assert np.isnan(y[T - 1]).all() and (T == 1 or np.isfinite(y[:T - 1]).all())
    if T > 1:
        _check_product(y[:T - 1], xq[:T - 1], xs[:T - 1], wq, ws)


def test_product_extreme_scales():
    # Scales of 1e30 and 1e-30 cancel: the product of the two is formed in FP32 without overflow on its own.
    rng = np.random.default_rng(6)
    xq, xs = f8.quantize(_acts(rng, 20, 256), 1)
    wq, ws = f8.quantize(_weights(rng, 130, 256), 128)
    xs, ws = (xs * np.float32(1e30)).astype(np.float32), (ws * np.float32(1e-30)).astype(np.float32)
    _check_product(_matmul(xq, xs, wq, ws), xq, xs, wq, ws)


def test_product_overflow_is_infinite():
    xq, wq = np.full((5, 128), 0x7E, np.uint8), np.full((40, 128), 0x7E, np.uint8)
    y = _matmul(xq, np.ones((5, 1), np.float32), wq, np.ones((1, 1), np.float32))
    assert np.isposinf(y).all()


@pytest.mark.parametrize("T,N,K", [(1, 4096, 2048), (77, 1001, 2064), (600, 1024, 1024)])
def test_product_repeats_bit_for_bit(T, N, K):
    rng = np.random.default_rng(K)
    xq, xs = f8.quantize(_acts(rng, T, K), 1)
    wq, ws = f8.quantize(_weights(rng, N, K), 128)
    a = _matmul(xq, xs, wq, ws)
    assert np.array_equal(a, _matmul(xq, xs, wq, ws))
    assert np.array_equal(a, _matmul(xq, xs, wq, ws, torch.cuda.Stream()))


def test_product_rows_do_not_depend_on_the_batch_neighbours():
    rng = np.random.default_rng(12)
    xq, xs = f8.quantize(_acts(rng, 300, 512), 1)
    wq, ws = f8.quantize(_weights(rng, 256, 512), 128)
    a = _matmul(xq, xs, wq, ws)
    xq2, xs2 = xq.copy(), xs.copy()
    xq2[1::2], xs2[1::2] = 0x7F, np.nan
    b = _matmul(xq2, xs2, wq, ws)
    assert np.array_equal(a[::2], b[::2]) and np.isnan(b[1::2]).all()


def test_product_beyond_32_bit_offsets():
    # 1,048,576 x 2064 codes (2.16e9) against 24 rows.
    T, N, K = 1 << 20, 24, 2064
    rng = np.random.default_rng(14)
    rows = [0, 5, 1_040_447, 1_040_448, 1_040_449, T - 1]
    xq, xs = f8.quantize(_acts(rng, len(rows), K), 1)
    wq, ws = f8.quantize(_weights(rng, N, K), 128)
    big = torch.full((T, K), 0x38, dtype=torch.uint8, device="cuda")
    bs = torch.ones((T, f8.nblocks(K)), device="cuda")
    big[rows] = torch.from_numpy(xq).cuda()
    bs[rows] = torch.from_numpy(xs).cuda()
    y = torch.zeros((T, N), dtype=torch.float16, device="cuda")
    work = torch.zeros(moe.moe_matmul_fp8_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    moe.moe_matmul_fp8(big.view(torch.float8_e4m3fn), bs, _codes(wq), torch.from_numpy(ws).cuda(), y, work)
    assert moe.moe_workspace_flags(work) == 0
    _check_product(y[rows].cpu().numpy(), xq, xs, wq, ws)


def test_product_refusals():
    f = torch.float8_e4m3fn
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda").view(f)
    s = torch.zeros(64, device="cuda")
    y = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.moe_matmul_fp8(z(4, 40), s, z(64, 40), s, y, ws)        # K not a multiple of 16
    with pytest.raises(ValueError):
        moe.moe_matmul_fp8(z(4, 32), s, z(64, 48), s, y, ws)
    with pytest.raises(ValueError):
        moe.moe_matmul_fp8(z(4, 32), s[:3], z(64, 32), s, y, ws)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_matmul_fp8(z(4, 32), s, z(64, 32), s, y, ws[:0])
    assert ei.value.status in (moe.MOE_ERR_CAPACITY, moe.MOE_ERR_ARG)
    with pytest.raises(moe.MoeError):
        moe.moe_matmul_fp8(z(4, 32), s, z(64, 32), s, y, ws[16:])   # workspace not 256-byte aligned
    with pytest.raises(moe.MoeError):
        moe.moe_matmul_fp8(z(4 * 32 + 16)[1:129].reshape(4, 32), s, z(64, 32), s, y, ws)
    moe.moe_matmul_fp8(z(0, 32), s, z(64, 32), s, y[:0], ws)        # no tokens: nothing to do


# ---- shared FFN -----------------------------------------------------------------
def _ffn_weights(rng, H, Is):
    out = []
    for r, c in ((Is, H), (Is, H), (H, Is)):
        out += list(f8.quantize(_weights(rng, r, c) * np.float16(2), 128))
    return out


def _ffn(x, w, stream=None):
    T, H = x.shape
    Is = w[0].shape[0]
    args = [_codes(a) if a.dtype == np.uint8 else torch.from_numpy(a).cuda() for a in w]
    xt = torch.from_numpy(x).cuda()
    y = torch.full((T, H), 777.0, dtype=torch.float16, device="cuda")
    ws = torch.zeros(moe.moe_shared_fp8_workspace_bytes(T, H, Is), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    moe.moe_shared_forward_fp8(xt, *args, y, ws, stream)
    torch.cuda.synchronize()
    assert moe.moe_workspace_flags(ws) == 0
    return y.cpu().numpy()


def _check_ffn(y, x, w):
    r = f8.shared_ffn(x, *w)
    g, u, h = r["g"], r["u"], r["h"]
    sig = 1.0 / (1.0 + np.exp(-g))
    dg, du = 2.0 ** -20 * r["ag"], 2.0 ** -20 * r["au"]
    dh = 1.1 * dg * np.abs(u) + np.abs(g * sig) * du + 2.0 ** -20 * np.abs(h)
    s = np.repeat(r["hs"], 128, 1)[:, :h.shape[1]]
    inv = np.where(s > 0, 1.0 / np.where(s > 0, s, 1.0), 0.0)
    # The block's scale moves with its largest element.
    T, Is = h.shape
    ds = np.zeros_like(h)
    for j in range(f8.nblocks(Is)):
        b = slice(j * 128, j * 128 + 128)
        i = np.argmax(np.abs(h[:, b]), 1)
        a = np.abs(h[np.arange(T), j * 128 + i])
        ds[:, b] = (dh[:, b].max(1) / np.where(a > 0, a, 1.0) + 2.0 ** -22)[:, None]
    v = h * inv
    dv = dh * inv + np.abs(v) * ds
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    moved = f8.encode(v - dv) != f8.encode(v + dv)
    wd = np.abs(r["wd"])
    tol = (2.0 ** -11 * np.abs(r["y"]) + 2.0 ** -20 * r["ay"] + 2.0 ** -25
           + (np.where(moved, step, 0.0) * s + np.abs(v) * s * ds) @ wd.T)
    err = np.abs(y.astype(np.float64) - r["y"])
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("T,H,Is", [(1, 64, 64), (1, 2048, 1024), (2, 256, 192), (4, 320, 4096), (16, 1024, 640),
                                    (31, 128, 1344), (64, 512, 128), (65, 2048, 320), (128, 192, 256), (130, 512, 320),
                                    (300, 1024, 1024), (513, 256, 512), (8, 512, 1344), (12, 64, 192), (9, 1088, 64),
                                    (3, 64, 704), (1024, 128, 192)])
def test_ffn_matches_oracle(T, H, Is):
    rng = np.random.default_rng(T + H + Is)
    x = rng.normal(size=(T, H)).astype(np.float16)
    w = _ffn_weights(rng, H, Is)
    _check_ffn(_ffn(x, w), x, w)


def test_ffn_config_shape_sampled():
    # The prefill configuration's shared FFN: 2048 tokens, H 2048, Is 4096.
    rng = np.random.default_rng(77)
    x = rng.normal(size=(2048, 2048)).astype(np.float16)
    w = []
    for r, c in ((4096, 2048), (4096, 2048), (2048, 4096)):
        w += list(_quantize(_weights(rng, r, c), 128))
    y = _ffn(x, w)
    rows = [0, 1, 127, 128, 255, 256, 1000, 1151, 2047]
    _check_ffn(y[rows], x[rows], w)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_ffn_zero_and_nonfinite_tokens(T):
    rng = np.random.default_rng(T)
    x = rng.normal(size=(T, 256)).astype(np.float16)
    w = _ffn_weights(rng, 256, 192)
    x[0] = 0
    y = _ffn(x, w)
    assert not y[0].any()
    if T > 1:
        _check_ffn(y[1:], x[1:], w)
        x[T // 2, 7] = np.nan
        y = _ffn(x, w)
        assert np.isnan(y[T // 2]).all()
        keep = [t for t in range(1, T) if t != T // 2]
        _check_ffn(y[keep], x[keep], w)


@pytest.mark.parametrize("Is", [64, 1024, 4608])
@pytest.mark.parametrize("T", [1, 9, 60, 300])
def test_ffn_vanishing_intermediate(T, Is):
    # Gate and up near 1e-20: h near 1e-40 and in places 0, where 448 / amax is
    # past FP32. y rounds to 0 in FP16, and nothing in it is NaN.
    rng = np.random.default_rng(T + Is)
    x = rng.normal(size=(T, 256)).astype(np.float16)
    w = _ffn_weights(rng, 256, Is)
    w[1], w[3] = np.full_like(w[1], 1e-22), np.full_like(w[3], 1e-22)
    w[2][::5] = 0
    assert np.abs(f8.shared_ffn(x, *w)["y"]).max() < 2.0 ** -25
    assert not _ffn(x, w).any()


@pytest.mark.parametrize("T,H,Is", [(4, 256, 192), (4, 256, 4608), (16, 256, 640), (60, 256, 320), (64, 2048, 512),
                                    (300, 256, 320), (2100, 256, 2304)])
@pytest.mark.parametrize("gate,up", [(-45.0, 1e17), (-60.0, 1e24), (-80.0, 1e33), (-1e5, 1e15), (-1e12, 1e8)])
def test_ffn_strongly_negative_gates(T, H, Is, gate, up):
    # silu(-45) is -1.3e-18 and silu(-1e5) is 0: with up large enough y shows it. Every gate here is near
    # `gate` and every up near `up`. A gate is off by up to 2^-20 of itself, h so by that much times |gate| (2e-4 at
    # most; where |gate| is 1e5 it is 0 all the same), and each element by one step of its code more: an eighth.
    rng = np.random.default_rng(T + Is)
    x = rng.uniform(0.9, 1.1, (T, H)).astype(np.float16)
    w = _ffn_weights(rng, H, Is)
    w[0], w[2] = np.full_like(w[0], 0xB8), np.full_like(w[2], 0x38)  # codes -1 and 1
    w[2][1::3] = 0xB8                                                # some ups negative
    w[1], w[3] = np.full_like(w[1], -gate / H), np.full_like(w[3], up / H)
    w[4] = w[4] & 0x7F                                               # W_d positive: sums do not cancel
    w[5] = w[5] / 32                                                 # y within FP16
    with np.errstate(over="ignore"):
        r = f8.shared_ffn(x, *w)
    assert (np.abs(r["y"]) > 1e-5).all() if gate > -1e4 else not r["y"].any()
    y = _ffn(x, w).astype(np.float64)
    assert np.isfinite(y).all()
    assert (np.abs(y - r["y"]) <= 0.13 * r["ay"] + 2.0 ** -11 * np.abs(r["y"]) + 2.0 ** -25).all()


@pytest.mark.parametrize("T", [1, 60, 300])
def test_ffn_repeats_bit_for_bit(T):
    rng = np.random.default_rng(T)
    x = rng.normal(size=(T, 512)).astype(np.float16)
    w = _ffn_weights(rng, 512, 1024)
    a = _ffn(x, w)
    assert np.array_equal(a, _ffn(x, w)) and np.array_equal(a, _ffn(x, w, torch.cuda.Stream()))


def test_ffn_equals_its_parts():
    # quantise, two products, SwiGLU in FP32 on the host, quantise, product.
    rng = np.random.default_rng(5)
    x = rng.normal(size=(70, 512)).astype(np.float16)
    w = _ffn_weights(rng, 512, 256)
    xq, xs = _quantize(x, 1)
    g, u = (f8.matmul(xq, xs, w[i], w[i + 1]) for i in (0, 2))
    hq, hs = f8.quantize((g / (1 + np.exp(-g)) * u).astype(np.float32), 1)
    parts = _matmul(hq, hs, w[4], w[5])
    y = _ffn(x, w)
    assert np.abs(parts.astype(float) - y).max() <= 2e-2 * np.abs(parts).max()


def test_ffn_workspace_serves_calls_of_other_sizes():
    # One workspace for a decode step, a prefill and a decode step again.
    rng = np.random.default_rng(21)
    H, Is = 256, 320
    w = _ffn_weights(rng, H, Is)
    args = [_codes(a) if a.dtype == np.uint8 else torch.from_numpy(a).cuda() for a in w]
    ws = torch.zeros(moe.moe_shared_fp8_workspace_bytes(400, H, Is), dtype=torch.uint8, device="cuda")
    assert ws.numel() >= moe.moe_shared_fp8_workspace_bytes(16, H, Is)
    for T in (1, 400, 5, 16, 90, 1):
        x = rng.normal(size=(T, H)).astype(np.float16)
        y = torch.empty((T, H), dtype=torch.float16, device="cuda")
        moe.moe_shared_forward_fp8(torch.from_numpy(x).cuda(), *args, y, ws)
        assert moe.moe_workspace_flags(ws) == 0
        _check_ffn(y.cpu().numpy(), x, w)


def test_calls_in_a_graph_repeat():
    # Quantisation, product and FFN captured once and replayed on new inputs in the same buffers.
    rng = np.random.default_rng(22)
    H, Is = 512, 256
    w = _ffn_weights(rng, H, Is)
    args = [_codes(a) if a.dtype == np.uint8 else torch.from_numpy(a).cuda() for a in w]
    for T in (2, 40, 300):
        x = torch.zeros((T, H), dtype=torch.float16, device="cuda")
        y = torch.empty_like(x)
        ws = torch.zeros(moe.moe_shared_fp8_workspace_bytes(T, H, Is), dtype=torch.uint8, device="cuda")
        moe.moe_shared_forward_fp8(x, *args, y, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_shared_forward_fp8(x, *args, y, ws)
        for _ in range(2):
            xn = rng.normal(size=(T, H)).astype(np.float16)
            x.copy_(torch.from_numpy(xn))
            g.replay()
            torch.cuda.synchronize()
            _check_ffn(y.cpu().numpy(), xn, w)


def test_ffn_refusals():
    f = torch.float8_e4m3fn
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda").view(f)
    s = torch.zeros(64, device="cuda")
    x = torch.zeros((4, 128), dtype=torch.float16, device="cuda")
    y = torch.zeros((4, 128), dtype=torch.float16, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.moe_shared_forward_fp8(x[:, :96].contiguous(), z(64, 96), s, z(64, 96), s, z(96, 64), s, y, ws)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_shared_forward_fp8(x, z(64, 128), s, z(64, 128), s, z(128, 64), s, y, ws[:256])
    assert ei.value.status == moe.MOE_ERR_CAPACITY
    with pytest.raises(ValueError):
        moe.moe_shared_forward_fp8(x, z(64, 128), s[:0], z(64, 128), s, z(128, 64), s, y, ws)
    with pytest.raises(TypeError):
        moe.moe_shared_forward_fp8(x.float(), z(64, 128), s, z(64, 128), s, z(128, 64), s, y, ws)
    moe.moe_shared_forward_fp8(x[:0], z(64, 128), s, z(64, 128), s, z(128, 64), s, y[:0], ws)


# ---- the layer --------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 12, 80])
def test_layer_with_scored_router_and_fp8_shared_path(T):
    # Scored routing, INT4 experts and the FP8 shared FFN as one layer; decode and grouped paths.
    shape, E, k, Is = (256, 128, 64), 16, 4, 320
    H = shape[0]
    rng = np.random.default_rng(T)
    lp = LayerPool(moe, 31, 0, shape, E)
    x = synth.activations(31, 1, T, H)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    bias = rng.permutation(np.linspace(-0.1, 0.1, E)).astype(np.float32)
    kw = dict(score="sigmoid", n_groups=4, top_groups=2, group_rank="top2", renorm=True, scale=2.5)
    w = _ffn_weights(rng, H, Is)
    ysh = _ffn(x, w)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    wt = torch.empty((T, k), dtype=torch.float32, device="cuda")
    y = torch.empty((T, H), dtype=torch.float16, device="cuda")
    ws = torch.zeros(moe.moe_forward_workspace_bytes(shape, T, k, E), dtype=torch.uint8, device="cuda")
    moe.moe_layer_forward_scored(shape, torch.from_numpy(x).cuda(), moe.moe_route_config(**kw),
                                 torch.from_numpy(logits).cuda(), k, torch.from_numpy(bias).cuda(), ids, wt, lp.pool,
                                 lp.slot_of, E, torch.from_numpy(ysh).cuda(), y, ws)
    assert moe.moe_workspace_flags(ws) == 0
    rid, rw, _ = f8.route_scored(logits, k, bias=bias, **kw)
    assert (f8.closest_call(logits, k, bias=bias, **kw) > 1e-6).all()
    assert np.array_equal(ids.cpu().numpy(), rid)
    ref = ysh.astype(np.float64)
    for t in range(T):
        for j in range(k):
            wg, wu, wd = moe_oracle.dequantize_expert(lp.arrays(int(rid[t, j])), shape[2])
            ref[t] += rw[t, j] * moe_oracle.expert_ffn(x[t].astype(np.float64), wg, wu, wd)
    err = np.abs(y.float().cpu().numpy() - ref).max()
    assert err <= 5e-3 * np.abs(ref).max(), err


@pytest.mark.parametrize("what", ["pairs", "grid", "alignment"])
def test_layer_scored_refuses_what_its_path_does_not_take_before_enqueueing(what):
    # More pairs than the grouped path sorts, or than the GEMV path's grid has rows; an output that the grouped
    # path cannot store 16 bytes at a time.
    shape, E, k = (256, 128, 64), 16, 8
    T = 64 if what == "alignment" else 65536 // k + (what == "pairs")
    path = moe.MOE_PATH_GEMV_UNFUSED if what == "grid" else moe.MOE_PATH_AUTO
    lp = LayerPool(moe, 31, 0, shape, E)
    x = torch.zeros((T, 256), dtype=torch.float16, device="cuda")
    ids = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    y = torch.zeros(T * 256 + 8, dtype=torch.float16, device="cuda")
    y = y[1:T * 256 + 1] if what == "alignment" else y[:T * 256]
    ws = torch.zeros(moe.moe_forward_workspace_bytes(shape, T, k, E, path), dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_layer_forward_scored(shape, x, moe.moe_route_config(), torch.zeros((T, E), device="cuda"), k, None, ids,
                                     torch.zeros((T, k), device="cuda"), lp.pool, lp.slot_of, E, None, y, ws, path)
    assert ei.value.status == (moe.MOE_ERR_ARG if what == "alignment" else moe.MOE_ERR_UNSUPPORTED)
    torch.cuda.synchronize()
    assert (ids == -9).all()


def test_layer_scored_refuses_before_enqueueing():
    shape, E, k = (256, 128, 64), 16, 4
    lp = LayerPool(moe, 31, 0, shape, E)
    x = torch.zeros((2, 256), dtype=torch.float16, device="cuda")
    ids = torch.full((2, k), -9, dtype=torch.int32, device="cuda")
    wt = torch.zeros((2, k), device="cuda")
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_layer_forward_scored(shape, x, moe.moe_route_config(), torch.zeros((2, E), device="cuda"), k, None, ids,
                                     wt, lp.pool, lp.slot_of, E, None, x.clone(),
                                     torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert ei.value.status == moe.MOE_ERR_CAPACITY and (ids == -9).all()
