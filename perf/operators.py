"""The measured cases of the FP8 and scored-routing operators.

Four operators of the serving path:
  route     moe_route_scored: softmax or sigmoid scores, a balance bias, expert
            groups, top-k, renormalised and scaled weights;
  quantize  moe_quantize_fp8: FP16 to E4M3 with one FP32 scale per block of
            1 x 128 (activations) or 128 x 128 (weights);
  matmul    moe_matmul_fp8: the block-scaled product of two such operands;
  ffn       moe_shared_forward_fp8: the shared SwiGLU FFN built from them.

`listed` and `draw` give cases, `prepare` what a program holds before the
call, `run` one pass (the plain form, or the library's calls when `own`),
`exact` the result in 64 bits, `work` the bytes and operations of one pass.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # One decoded token of a model with 256 experts in 8 groups: sigmoid
        # scores, balance bias, four groups by their two best, top-8.
        dict(name="route-token", op="route", T=1, E=256, k=8, G=8, top_g=4, rank="top2", score="sigmoid",
             bias=True, renorm=True, scale=2.5, half=False, masked=False),
        # A batch of 256 tokens over the 512-expert top-10 stack, softmax with
        # a bias, logits straight from an FP16 gate.
        dict(name="route-batch", op="route", T=256, E=512, k=10, G=1, top_g=1, rank="max", score="softmax",
             bias=True, renorm=True, scale=1.0, half=True, masked=False),
        # 60 experts, top-4, odd token count, some experts masked out per token
        # (some tokens have none left), groups by their best, no bias.
        dict(name="route-odd", op="route", T=1021, E=60, k=4, G=6, top_g=3, rank="max", score="softmax",
             bias=False, renorm=False, scale=1.0, half=False, masked=True),
        # A long prefill through the grouped sigmoid router.
        dict(name="route-prefill", op="route", T=32768, E=256, k=8, G=8, top_g=4, rank="top2", score="sigmoid",
             bias=True, renorm=True, scale=2.5, half=False, masked=False),
        # Activations of a long prefill.
        dict(name="quantize-rows", op="quantize", rows=8192, cols=4096, block_rows=1),
        # Weights laid out once at load time; rows that end inside a block.
        dict(name="quantize-weight", op="quantize", rows=4040, cols=2048, block_rows=128),
        # One decoded token: bound by the weight bytes and the launch.
        dict(name="matmul-token", op="matmul", T=1, N=4096, K=2048),
        # A decode batch against a ragged matrix (N odd, K ends inside a block).
        dict(name="matmul-odd", op="matmul", T=77, N=1001, K=2064),
        # A prefill projection.
        dict(name="matmul-prefill", op="matmul", T=2048, N=4096, K=2048),
        # The largest projection.
        dict(name="matmul-large", op="matmul", T=8192, N=8192, K=4096),
        # The shared FFN of one decoded token, and of the 2048-token prefill.
        dict(name="ffn-token", op="ffn", T=1, H=2048, Is=4096),
        dict(name="ffn-prefill", op="ffn", T=2048, H=2048, Is=4096),
    ]


def _size(rng, lo, hi, unit=1):
    """A multiple of `unit`, spread over the logarithm; 3072 is no size of this repository."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return unit * (n if n * unit != 3072 else n - 1)


def draw(rng):
    op = rng.choice(["route", "quantize", "matmul", "ffn"])
    if op == "route":
        G = rng.choice([1, 1, 2, 4, 6, 8, 16])
        E = _size(rng, 8 // G + 1, 1024 // G, G)
        top_g = rng.randint(1, G)
        k = rng.randint(1, min(16, top_g * (E // G)))
        T = min(_size(rng, 1, 32768), (32768 * 256) // E)
        return dict(op="route", T=T, E=E, k=k, G=G, top_g=top_g, rank=rng.choice(["max", "top2"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 1.5, 2.5]), half=rng.random() < 0.3, masked=rng.random() < 0.25)
    if op == "quantize":
        return dict(op="quantize", rows=_size(rng, 1, 8192), cols=_size(rng, 1, 256, 16),
                    block_rows=rng.choice([1, 1, 128]))
    if op == "matmul":
        K = _size(rng, 4, 512, 16)
        N = _size(rng, 8, 8192)
        T = min(_size(rng, 1, 8192), (8192 * 8192 * 4096) // (N * K))
        return dict(op="matmul", T=T, N=N, K=K)
    H, Is = _size(rng, 1, 64, 64), _size(rng, 1, 96, 64)
    return dict(op="ffn", T=min(_size(rng, 1, 4096), (2048 * 2048 * 4096) // (H * Is)), H=H, Is=Is)


def _blocks(n):
    return -(-n // 128)


def work(case):
    c = case
    if c["op"] == "route":
        e = 2 if c["half"] else 4
        return {"bytes": c["T"] * c["E"] * e + (4 * c["E"] if c["bias"] else 0) + 8 * c["T"] * c["k"],
                "flops": 6 * c["T"] * c["E"]}
    if c["op"] == "quantize":
        br = c["block_rows"]
        return {"bytes": 3 * c["rows"] * c["cols"] + 4 * -(-c["rows"] // br) * _blocks(c["cols"]),
                "flops": 3 * c["rows"] * c["cols"]}
    if c["op"] == "matmul":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": (T + N) * K + 4 * (T + _blocks(N)) * _blocks(K) + 2 * T * N, "flops": 2 * T * N * K}
    T, H, Is = c["T"], c["H"], c["Is"]
    return {"bytes": 3 * H * Is + 12 * _blocks(H) * _blocks(Is) + 4 * T * H, "flops": 6 * T * H * Is}


# ---- inputs -----------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _logits(c, g, rows, popularity):
    l = 1.5 * torch.randn((rows, c["E"]), generator=g, device=DEV) + popularity
    if c["half"]:
        l = l.half()
    if c["masked"]:
        l = l.masked_fill(torch.rand((rows, c["E"]), generator=g, device=DEV) < 0.3, -math.inf)
    return l


def _settled(c, logits, bias):
    """Rows whose choice does not hinge on the last bits of an exponential:
    in 64 bits, no two of the computed values that decide the order are within
    2e-6 of each other. Where they are, FP32 may order them either way, and both
    answers are right. (Without a bias the logits themselves order the
    experts, exactly, ties included.)"""
    value, group = _order_values(c, logits.double(), None if bias is None else bias.double())
    ok = torch.ones(logits.shape[0], dtype=torch.bool, device=DEV)
    if group is not None and c["top_g"] < c["G"] and (bias is not None or c["rank"] == "top2"):
        gs = group.sort(1, descending=True)[0]
        ok &= ~((gs[:, c["top_g"] - 1] - gs[:, c["top_g"]]).abs() < 2e-6)
    if bias is not None:
        vs = value.sort(1, descending=True)[0][:, :c["k"] + 1]
        ok &= ~((vs[:, :-1] - vs[:, 1:]).abs() < 2e-6).any(1)
    return ok


def _prepare_route(c, seed):
    g = _gen(seed)
    T, E, k = c["T"], c["E"], c["k"]
    popularity = 0.5 * torch.randn((E,), generator=g, device=DEV)
    # The bias of a balanced router: small, its own value for each expert.
    bias = (torch.linspace(-0.1, 0.1, E, device=DEV)[torch.randperm(E, generator=g, device=DEV)]
            if c["bias"] else None)
    logits = _logits(c, g, T, popularity)
    todo = torch.arange(T, device=DEV)
    while todo.numel():
        todo = todo[~_settled(c, logits[todo], bias)]
        logits[todo] = _logits(c, g, todo.numel(), popularity)
    if c["masked"]:
        logits[T // 2::97] = -math.inf  # tokens whose mask leaves no expert
    st = dict(c=c, logits=logits, bias=bias, ids=torch.empty((T, k), dtype=torch.int32, device=DEV),
              w=torch.empty((T, k), dtype=torch.float32, device=DEV))
    if own:  # the router's settings, made once per model
        st["cfg"] = _moe().moe_route_config(score=c["score"], n_groups=c["G"], top_groups=c["top_g"],
                                            group_rank=c["rank"], renorm=c["renorm"], scale=c["scale"])
    return st


def _activations(g, rows, cols):
    # N(0, 1) with a few outlier channels, as a norm's output has.
    x = torch.randn((rows, cols), generator=g, device=DEV)
    return (x * torch.where(torch.rand((cols,), generator=g, device=DEV) < 0.01, 12.0, 1.0)).half()


def _weights(g, rows, cols):
    s = 0.02 * torch.exp(0.3 * torch.randn((rows, 1), generator=g, device=DEV))
    return (torch.randn((rows, cols), generator=g, device=DEV) * s).half()


def prepare(case, seed):
    c = dict(case)
    if c["op"] == "route":
        return _prepare_route(c, seed)
    g = _gen(seed)
    st = dict(c=c)
    if c["op"] == "quantize":
        x = _activations(g, c["rows"], c["cols"]) if c["block_rows"] == 1 else _weights(g, c["rows"], c["cols"])
        if c["rows"] > 2:
            x[c["rows"] // 2, :128] = 0  # a block of zeros
        st["x"] = x
        st["q"] = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=DEV)
        st["s"] = torch.empty((-(-c["rows"] // c["block_rows"]), _blocks(c["cols"])), device=DEV)
    elif c["op"] == "matmul":
        st["xq"], st["xs"] = _quantize(_activations(g, c["T"], c["K"]), 1)
        st["wq"], st["ws"] = _quantize(_weights(g, c["N"], c["K"]), 128)
        st["y"] = torch.empty((c["T"], c["N"]), dtype=torch.float16, device=DEV)
        if own:  # the workspace that a program keeps
            st["work"] = torch.zeros(_moe().moe_matmul_fp8_workspace_bytes(c["T"], c["N"], c["K"]), dtype=torch.uint8,
                                     device=DEV)
    else:
        T, H, Is = c["T"], c["H"], c["Is"]
        st["x"] = torch.randn((T, H), generator=g, device=DEV).half()
        for n, (r, k) in dict(g=(Is, H), u=(Is, H), d=(H, Is)).items():
            st["w" + n], st["s" + n] = _quantize(_weights(g, r, k), 128)
        st["y"] = torch.empty((T, H), dtype=torch.float16, device=DEV)
        if own:  # the workspace that a program keeps
            st["work"] = torch.zeros(_moe().moe_shared_fp8_workspace_bytes(T, H, Is), dtype=torch.uint8, device=DEV)
    return st


# ---- plain forms --------------------------------------------------------------
def _moe():
    from int4_routed_expert_moe_gb300 import moe
    return moe


def _scores(c, l):
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.max(1, keepdim=True)[0])
    return e / e.sum(1, keepdim=True)


def _order_values(c, l, bias):
    """What orders the experts of each token (-inf: not to be chosen), and the
    groups' values (None without groups). Without a bias the logits order
    them: both scores grow with the logit."""
    T, E, G = l.shape[0], c["E"], c["G"]
    live = l > -math.inf
    s = _scores(c, l)
    if bias is None:
        value = l + 0.0
    else:
        s = s + bias
        value = s
    value = torch.where(live, value, -math.inf)
    if G == 1:
        return value, None
    if c["rank"] == "max" or E == G:
        group = value.view(T, G, E // G).max(2)[0]
    else:
        top = torch.where(live, s, -math.inf).view(T, G, E // G).sort(2, descending=True)[0][:, :, :2]
        group = top[:, :, 0] + torch.where(top[:, :, 1] > -math.inf, top[:, :, 1], 0.0)
    kept = torch.zeros((T, G), dtype=torch.bool, device=l.device)
    kept.scatter_(1, group.sort(dim=1, descending=True, stable=True)[1][:, :c["top_g"]], True)
    return torch.where(kept.repeat_interleave(E // G, 1), value, -math.inf), group


def _route(c, logits, bias):
    l = logits.float()
    bad = (torch.isnan(l) | (l == math.inf)).any(1, keepdim=True) | ~(l > -math.inf).any(1, keepdim=True)
    value, _ = _order_values(c, l, bias)
    value, order = value.sort(dim=1, descending=True, stable=True)
    value, order = value[:, :c["k"]], order[:, :c["k"]]
    chosen = (value > -math.inf) & ~bad
    w = torch.where(chosen, _scores(c, l).gather(1, order), 0.0)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return torch.where(chosen, order, -1).int(), w * c["scale"]


def _quantize(x, block_rows):
    """E4M3 codes and FP32 scales of blocks of block_rows x 128: s = amax / 448, q = x * (448 / amax)."""
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), _blocks(cols)
    p = torch.nn.functional.pad(x.float(), (0, 128 * cb - cols, 0, block_rows * rb - rows))
    p = p.view(rb, block_rows, cb, 128)
    amax = p.abs().amax((1, 3))
    inv = torch.where(amax > 0, E4M3_MAX / amax, 0.0)
    q = (p * inv[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(rb * block_rows, 128 * cb)[:rows, :cols].contiguous(), amax / E4M3_MAX


def _widen(q, s, block_rows):
    """The FP32 values that codes and scales stand for."""
    rows, cols = q.shape
    s = s.repeat_interleave(128, 1)[:, :cols]
    return q.float() * (s if block_rows == 1 else s.repeat_interleave(128, 0)[:rows])


def _product(xq, xs, wq, ws):
    return _widen(xq, xs, 1) @ _widen(wq, ws, 128).t()


def run(state):
    c = state["c"]
    if c["op"] == "route":
        if own:
            _moe().moe_route_scored(state["cfg"], state["logits"], c["k"], state["bias"], state["ids"], state["w"])
            return {"ids": state["ids"], "weights": state["w"]}
        ids, w = _route(c, state["logits"], state["bias"])
        return {"ids": ids, "weights": w}
    if c["op"] == "quantize":
        if own:
            _moe().moe_quantize_fp8(state["x"], state["q"], state["s"], c["block_rows"])
            return {"q": state["q"], "scales": state["s"]}
        q, s = _quantize(state["x"], c["block_rows"])
        return {"q": q, "scales": s}
    if c["op"] == "matmul":
        if own:
            _moe().moe_matmul_fp8(state["xq"], state["xs"], state["wq"], state["ws"], state["y"], state["work"])
            return state["y"]
        return _product(state["xq"], state["xs"], state["wq"], state["ws"]).half()
    if own:
        _moe().moe_shared_forward_fp8(state["x"], state["wg"], state["sg"], state["wu"], state["su"], state["wd"],
                                      state["sd"], state["y"], state["work"])
        return state["y"]
    xq, xs = _quantize(state["x"], 1)
    gate = _product(xq, xs, state["wg"], state["sg"])
    h = gate / (1.0 + torch.exp(-gate)) * _product(xq, xs, state["wu"], state["su"])
    hq, hs = _quantize(h, 1)
    return _product(hq, hs, state["wd"], state["sd"]).half()


# ---- 64 bits ------------------------------------------------------------------
def _exact_route(c, logits, bias):
    l = logits.cpu().numpy().astype(np.float64)
    b = np.zeros(c["E"]) if bias is None else bias.cpu().numpy().astype(np.float64)
    T, E, G, k = l.shape[0], c["E"], c["G"], c["k"]
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    some = np.isfinite(l).any(1)
    l = l[some]
    n = l.shape[0]
    if n:
        if c["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - l.max(1)[:, None])
            s = s / s.sum(1)[:, None]
        off = np.isneginf(l)
        key = np.where(off, -np.inf, l if bias is None else s + b)
        if G > 1:
            per = E // G
            if c["rank"] == "max" or per == 1:
                gv = key.reshape(n, G, per).max(2)
            else:
                t = np.sort(np.where(off, -np.inf, s + b).reshape(n, G, per), 2)[:, :, -2:]
                gv = t[:, :, 1] + np.where(np.isneginf(t[:, :, 0]), 0.0, t[:, :, 0])
            drop = np.argsort(-gv, 1, kind="stable")[:, c["top_g"]:]
            out = np.zeros((n, G), bool)
            np.put_along_axis(out, drop, True, 1)
            key = np.where(np.repeat(out, per, 1), -np.inf, key)
        top = np.argsort(-key, 1, kind="stable")[:, :k]
        dead = np.isneginf(np.take_along_axis(key, top, 1))
        ws = np.where(dead, 0.0, np.take_along_axis(s, top, 1))
        if c["renorm"]:
            ws = ws / (ws.sum(1)[:, None] + 1e-20)
        ids[some], w[some] = np.where(dead, -1, top), ws * c["scale"]
    return {"ids": ids, "weights": w}


def _exact_codes(v):
    """Nearest E4M3 value of each |v| <= 448, ties to even: 3 bits after the leading one, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quantize(x, br):
    """Codes' values and scales in 64 bits, block column by block column."""
    rows, cols = x.shape
    q = torch.zeros((rows, cols), dtype=torch.float64, device=x.device)
    s = torch.zeros((-(-rows // br), _blocks(cols)), dtype=torch.float64, device=x.device)
    for j in range(_blocks(cols)):
        col = x[:, 128 * j:128 * j + 128].double()
        m = col.abs().max(1)[0]
        m = torch.stack([p.max() for p in m.split(br)]) if br > 1 else m
        s[:, j] = m / E4M3_MAX
        each = m.repeat_interleave(br)[:rows, None]
        q[:, 128 * j:128 * j + 128] = _exact_codes(torch.where(each > 0, col * E4M3_MAX / each, 0.0))
    return q, s


def _exact_product(xq, xs, wq, ws):
    """Sum over blocks of 128 of scale * scale * (codes' product)."""
    y = torch.zeros((xq.shape[0], wq.shape[0]), dtype=torch.float64, device=xq.device)
    for j in range(xs.shape[1]):
        a = xq[:, 128 * j:128 * j + 128].double() * xs[:, j:j + 1].double()
        b = wq[:, 128 * j:128 * j + 128].double()
        y += (a @ b.t()) * ws[:, j].double().repeat_interleave(128)[:wq.shape[0]]
    return y


def exact(case, seed):
    st = prepare(case, seed)
    c = st["c"]
    if c["op"] == "route":
        return _exact_route(c, st["logits"], st["bias"])
    if c["op"] == "quantize":
        q, s = _exact_quantize(st["x"], c["block_rows"])
        return {"q": q, "scales": s}
    if c["op"] == "matmul":
        return _exact_product(st["xq"], st["xs"], st["wq"], st["ws"])
    xq, xs = _exact_quantize(st["x"], 1)
    gate = _exact_product(xq, xs, st["wg"], st["sg"])
    up = _exact_product(xq, xs, st["wu"], st["su"])
    hq, hs = _exact_quantize(gate * up / (1.0 + torch.exp(-gate)), 1)
    return _exact_product(hq, hs, st["wd"], st["sd"])
