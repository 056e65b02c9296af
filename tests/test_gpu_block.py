"""A whole MoE block in one call: the same bits as its parts called one by one, close to the oracle, with its
router's balance loss and gradient behind it (needs a GB300)."""
import numpy as np
import pytest
import torch

from int4_routed_expert_moe_gb300 import synth
from oracle import block_oracle as bo
from oracle import fp8_oracle, moe_oracle
from tests._lib import binding
from tests.gpu_util import LayerPool

pytestmark = pytest.mark.gpu

moe = binding() if torch.cuda.is_available() else None
SHAPE, E, K = (256, 128, 64), 16, 4


@pytest.fixture(scope="module")
def pool():
    return LayerPool(moe, synth.BASE_SEED, 0, SHAPE, E)


class Model:
    def __init__(self, pool, shared, post, kind="rms", score="sigmoid", seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        H, half = SHAPE[0], torch.float16
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")
        vec = lambda m: (m + 0.2 * rand(H)).to(half)
        self.pool, self.Is = pool, 128 if shared else 0
        self.norm = moe.moe_norm_config(kind, 1e-5)
        self.route = moe.moe_route_config(score, 4, 2, "top2", True, 1.5)
        self.norm_w, self.norm_b = vec(1.0), vec(0.0) if kind == "layer" else None
        self.post_w, self.post_b = (vec(1.0), vec(0.0) if kind == "layer" else None) if post else (None, None)
        self.gate_w, self.gate_b = (rand(E, H) * 0.1).to(half), 0.1 * rand(E)
        self.bias = torch.linspace(-0.1, 0.1, E, device="cuda")
        w = lambda r, c: (rand(r, c) * c ** -0.5).to(half)
        self.shared = (w(self.Is, H), w(self.Is, H), w(H, self.Is)) if shared else None
        self.block = moe.moe_block_config(SHAPE, K, self.norm, self.norm_w, self.gate_w, self.route, pool.pool,
                                          pool.slot_of, E, self.norm_b, self.gate_b, self.bias, self.shared, self.post_w,
                                          self.post_b, 0.75, 1.25)

    def workspace(self, T):
        return torch.zeros(moe.moe_block_workspace_bytes(self.block, T), dtype=torch.uint8, device="cuda")

    def parts(self, h):
        """The same by the separate calls; returns h, ids, weights, logits, y."""
        T, H = h.shape
        new = lambda *s, d=torch.float16: torch.empty(s, dtype=d, device="cuda")
        zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
        n, logits, y, ids, w = new(T, H), new(T, E, d=torch.float32), new(T, H), new(T, K, d=torch.int32), new(T, K, d=torch.float32)
        moe.moe_norm(self.norm, h, self.norm_w, self.norm_b, n)
        moe.moe_linear(n, self.gate_w, self.gate_b, logits, zeros(moe.moe_linear_workspace_bytes(T, E, H)))
        ysh = None
        if self.shared is not None:
            ysh = new(T, H)
            moe.moe_shared_forward(n, *self.shared, ysh, zeros(moe.moe_shared_workspace_bytes(T, H, self.Is)))
        moe.moe_layer_forward_scored(SHAPE, n, self.route, logits, K, self.bias, ids, w, self.pool.pool, self.pool.slot_of,
                                     E, ysh, y, zeros(moe.moe_forward_workspace_bytes(SHAPE, T, K, E)))
        out = torch.empty_like(h)
        moe.moe_norm_residual(self.norm, y, h, out, self.post_w, self.post_b, None, 0.75, 1.25)
        return out, ids, w, logits, n, y


def _stream(T, f32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T)
    return (torch.randn((T, SHAPE[0]), generator=g, device="cuda") * 2).to(torch.float32 if f32 else torch.float16)


def _out(T):
    return torch.full((T, K), -9, dtype=torch.int32, device="cuda"), torch.full((T, K), 9.0, device="cuda")


@pytest.mark.parametrize("shared,post,kind,f32", [(False, False, "rms", True), (True, False, "rms", False),
                                                  (True, True, "layer", True), (False, True, "rms", False)])
@pytest.mark.parametrize("T", [1, 3, 16, 17, 130, 700])
def test_same_bits_as_the_parts(pool, T, shared, post, kind, f32):
    m = Model(pool, shared, post, kind)
    h = _stream(T, f32)
    want = m.parts(h)
    ids, w = _out(T)
    logits, ws = torch.full((T, E), 9.0, device="cuda"), m.workspace(T)
    got = h.clone()
    moe.moe_block_forward(m.block, got, ids, w, ws, logits)
    assert all(torch.equal(a, b) for a, b in zip((got, ids, w, logits), want))
    assert moe.moe_workspace_flags(ws) == 0
    got = h.clone()
    moe.moe_block_forward(m.block, got, ids, w, ws)  # logits in the workspace
    assert torch.equal(got, want[0]) and torch.equal(ids, want[1])


def test_against_the_oracle(pool):
    T = 9
    m = Model(pool, True, True)
    h = _stream(T, True)
    x = h.double().cpu().numpy()
    num = lambda t: t.double().cpu().numpy()
    n, _ = bo.norm(x, num(m.norm_w), None, "rms", 1e-5)
    n16 = n.astype(np.float16)
    logits, _ = bo.linear(n16, num(m.gate_w), num(m.gate_b))
    got, ids, w, lg, gn, gy = m.parts(h)
    assert np.abs(num(gn) - n).max() <= 2.0 ** -10 * np.abs(n).max()
    # From the FP16 n on: a rounding boundary may fall the other way, 2^-11 of a few of 256 terms.
    assert np.abs(num(lg) - logits).max() <= 2.0 ** -8
    rid, rw, _ = fp8_oracle.route_scored(lg.cpu().numpy(), K, bias=m.bias.cpu().numpy(), score="sigmoid", n_groups=4, top_groups=2,
                                         group_rank="top2", renorm=True, scale=1.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    nn = gn.cpu().numpy()
    y = moe_oracle.shared_ffn(nn, *[t.cpu().numpy() for t in m.shared])
    for t in range(T):
        for j in range(K):
            mats = moe_oracle.dequantize_expert(pool.arrays(int(rid[t, j])), SHAPE[2])
            y[t] += rw[t, j] * moe_oracle.expert_ffn(nn[t], *mats)
    assert np.abs(num(gy) - y).max() <= 5e-3 * np.abs(y).max()
    a, _ = bo.norm(num(gy), num(m.post_w), None, "rms", 1e-5)
    assert np.abs(num(got) - (1.25 * x + 0.75 * a)).max() <= 2.0 ** -17 * np.abs(x).max()
    block_h, (bi, bw) = h.clone(), _out(T)
    moe.moe_block_forward(m.block, block_h, bi, bw, m.workspace(T))
    assert torch.equal(block_h, got)


def test_one_workspace_for_several_batch_sizes_graph_and_stream(pool):
    m = Model(pool, True, True)
    sizes = (700, 1, 130, 16, 5, 17, 1, 700)
    ws = torch.zeros(max(moe.moe_block_workspace_bytes(m.block, T) for T in sizes), dtype=torch.uint8, device="cuda")
    for T in sizes:
        h, (ids, w) = _stream(T, True), _out(T)
        want = m.parts(h)
        moe.moe_block_forward(m.block, h, ids, w, ws)
        assert torch.equal(h, want[0]) and torch.equal(ids, want[1]), T
        assert moe.moe_workspace_flags(ws) == 0, T
    T = 6
    h0, (ids, w) = _stream(T, True), _out(T)
    h = h0.clone()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        moe.moe_block_forward(m.block, h, ids, w, ws)
        moe.moe_block_forward(m.block, h, ids, w, ws)
    want = m.parts(m.parts(h0)[0])
    for _ in range(3):
        h.copy_(h0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(ids, want[1])


@pytest.mark.parametrize("T", [2, 40])
def test_error_words_are_collected(pool, T):
    m = Model(pool, True, False)
    h, (ids, w), ws = _stream(T, True), _out(T), m.workspace(T)
    bad = pool.slot_of.clone()
    bad[:] = E + 3  # every slot outside the pool
    b = moe.moe_block_config(SHAPE, K, m.norm, m.norm_w, m.gate_w, m.route, pool.pool, bad, E, shared=m.shared)
    moe.moe_block_forward(b, h, ids, w, ws)
    assert moe.moe_workspace_flags(ws) == 1
    moe.moe_block_forward(m.block, h, ids, w, ws)  # sticky
    assert moe.moe_workspace_flags(ws) == 1
    moe.moe_workspace_clear_flags(ws)
    moe.moe_block_forward(m.block, h, ids, w, ws)
    assert moe.moe_workspace_flags(ws) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_training_step_of_the_router(pool, score):
    # Block forward, balance loss over two sequences and padding, gradient of the logits: against differences of
    # the whole chain's loss along the gate's bias (the picks, and so f, stay as they are).
    T, off = 50, np.array([0, 20, 47], np.int32)
    m = Model(pool, False, False, score=score)
    h0, (ids, w), ws = _stream(T, True), _out(T), m.workspace(T)
    logits, o = torch.empty((T, E), device="cuda"), torch.from_numpy(off).cuda()
    cfg = moe.moe_balance_config(score, 1.0)
    counts, tokens = torch.empty((2, E), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    loss, d = torch.empty(1, device="cuda"), torch.zeros((T, E), device="cuda")
    work = torch.zeros(moe.moe_balance_workspace_bytes(T, E, 2), dtype=torch.uint8, device="cuda")
    moe.moe_block_forward(m.block, h0.clone(), ids, w, ws, logits)
    moe.moe_balance_loss(cfg, logits, ids, o, counts, tokens, None, loss, work)
    moe.moe_balance_loss_backward(cfg, logits, K, o, counts, tokens, None, d)
    assert counts.sum() == 47 * K and tokens.tolist() == [20, 27] and (d[47:] == 0).all()
    keep, base, step = ids.clone(), m.gate_b.clone(), 0.05
    for e in (0, 7, 15):
        v = []
        for s in (step, -step):
            m.gate_b.copy_(base)
            m.gate_b[e] += s
            moe.moe_block_forward(m.block, h0.clone(), ids, w, ws, logits)
            moe.moe_balance_loss(cfg, logits, keep, o, counts, tokens, None, loss, work)
            v.append(float(loss))
        m.gate_b.copy_(base)
        want = float(d[:, e].sum())
        # Third derivatives of a mean of probabilities are below 1; losses carry 2^-20.
        f_max = float((counts.float() * E / K / tokens[:, None]).max())
        assert abs((v[0] - v[1]) / (2 * step) - want) <= f_max * step ** 2 / 6 + (abs(v[0]) + abs(v[1])) * 2.0 ** -21 / step


def test_refusals(pool):
    m = Model(pool, True, False)
    h, (ids, w), ws = _stream(4, True), _out(4), m.workspace(4)
    with pytest.raises(ValueError):
        moe.moe_block_forward(m.block, h[:, :128].contiguous(), ids, w, ws)
    with pytest.raises(ValueError):
        moe.moe_block_forward(m.block, h, ids[:2], w, ws)
    with pytest.raises(moe.MoeError):
        moe.moe_block_forward(m.block, h, ids, w, ws[:1024])
    with pytest.raises(TypeError):
        moe.moe_block_forward(m.block, h.double(), ids, w, ws)
    with pytest.raises(ValueError):
        moe.moe_block_config(SHAPE, K, m.norm, m.norm_w, m.gate_w.t().contiguous(), m.route, pool.pool, pool.slot_of, E)
    with pytest.raises(ValueError):
        moe.moe_block_config(SHAPE, K, m.norm, m.norm_w, m.gate_w, m.route, pool.pool, pool.slot_of, E,
                             shared=(m.shared[0], m.shared[1], m.shared[2].t().contiguous()))
    b = moe.moe_block_config(SHAPE, K, m.norm, m.norm_w, m.gate_w, m.route, pool.pool, pool.slot_of, E, norm_b=m.norm_w)
    with pytest.raises(moe.MoeError):  # an RMS norm has no bias
        moe.moe_block_forward(b, h, ids, w, ws)
    moe.moe_block_forward(m.block, h[:0], ids[:0], w[:0], ws)


def test_a_refused_batch_leaves_the_buffers_as_they_were():
    # 32 picks of inter 4096 exceed the GEMV path's shared memory; the same block serves batches of the grouped path.
    shape, experts, k = (256, 4096, 64), 64, 32
    one = torch.zeros(moe.moe_expert_block_bytes(shape), dtype=torch.uint8, device="cuda")
    slot_of = torch.zeros(experts, dtype=torch.int32, device="cuda")
    half = lambda *s: torch.ones(s, dtype=torch.float16, device="cuda")
    b = moe.moe_block_config(shape, k, moe.moe_norm_config(), half(256), half(experts, 256), moe.moe_route_config(), one,
                             slot_of, 1, shared=(half(128, 256), half(128, 256), half(256, 128)))
    ws = torch.zeros(moe.moe_block_workspace_bytes(b, 20), dtype=torch.uint8, device="cuda")
    for T, refused in ((2, True), (20, False)):
        h, logits = torch.full((T, 256), 2.0, device="cuda"), torch.full((T, experts), 9.0, device="cuda")
        ids, w = torch.full((T, k), -9, dtype=torch.int32, device="cuda"), torch.full((T, k), 9.0, device="cuda")
        before = ws.clone()
        if not refused:
            moe.moe_block_forward(b, h, ids, w, ws, logits)
            assert (ids >= 0).all() and (logits != 9.0).all() and moe.moe_workspace_flags(ws) == 0
            continue
        with pytest.raises(moe.MoeError) as e:
            moe.moe_block_forward(b, h, ids, w, ws, logits)
        assert e.value.status == moe.MOE_ERR_UNSUPPORTED
        torch.cuda.synchronize()
        assert (h == 2.0).all() and (logits == 9.0).all() and (ids == -9).all() and (w == 9.0).all()
        assert torch.equal(ws, before)
