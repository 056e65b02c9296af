"""The measured cases of the operators around the routed layer.

Three operators, one of them with its gradient:
  norm      moe_norm_residual: what a block adds to the residual stream (after
            a norm of its own, times a gate and a scale), and the next block's
            norm of the sum, as FP16 and as FP8 codes; moe_norm: the norm alone;
  linear    moe_linear: y = act(x W^T + b) + residual, FP16 operands;
  balance   moe_balance_loss: the router's balance loss and per-expert counts,
            by sequence, and moe_balance_loss_backward: its gradient.

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
        # Between two blocks of one decoded token: the residual sum and the next norm.
        dict(name="norm-token", op="norm", T=1, H=2048, kind="rms", stream32=False, branch=True, post=False,
             gate="none", half=True, fp8=False, offset=0.0),
        # A ragged batch of a model that also norms what a block gives, with a gate per token (a
        # shared path's), over an FP32 residual stream; weights stored around zero.
        dict(name="norm-both-odd", op="norm", T=1021, H=2008, kind="rms", stream32=True, branch=True, post=True,
             gate="token", half=True, fp8=False, offset=1.0),
        # A long prefill in front of an FP8 projection: FP16 for the router's gate, codes for the product.
        dict(name="norm-prefill", op="norm", T=8192, H=4096, kind="rms", stream32=True, branch=True, post=False,
             gate="channel", half=True, fp8=True, offset=0.0),
        # The router's gate for one decoded token: FP32 logits of 256 experts.
        dict(name="linear-gate-token", op="linear", T=1, N=256, K=2048, act="none", bias=False, residual=False, out32=True),
        # A decode batch's output projection with its residual.
        dict(name="linear-batch", op="linear", T=16, N=2048, K=4096, act="none", bias=False, residual=True, out32=False),
        # An odd batch against a ragged matrix, bias and activation.
        dict(name="linear-odd", op="linear", T=77, N=1001, K=2064, act="gelu", bias=True, residual=False, out32=False),
        # The router's gate for a long prefill.
        dict(name="linear-gate-prefill", op="linear", T=8192, N=256, K=2048, act="none", bias=True, residual=False,
             out32=True),
        # The largest projection, with bias, activation and residual.
        dict(name="linear-large", op="linear", T=8192, N=8192, K=4096, act="silu", bias=True, residual=True, out32=False),
        # A small training batch of a 64-expert top-8 router, one sequence.
        dict(name="balance-batch", op="balance", back=False, T=256, E=64, k=8, S=1, score="softmax", half=False,
             masked=False, padded=False),
        # Sixteen ragged sequences through a 256-expert sigmoid router.
        dict(name="balance-prefill", op="balance", back=False, T=32768, E=256, k=8, S=16, score="sigmoid", half=False,
             masked=False, padded=False),
        # The gradient for 60 experts behind an FP16 gate: seven sequences (one empty), experts masked
        # per token (some tokens have none), a padded batch.
        dict(name="balance-back-odd", op="balance", back=True, T=4093, E=60, k=4, S=7, score="sigmoid", half=True,
             masked=True, padded=True),
        # The gradient of a long batch.
        dict(name="balance-back", op="balance", back=True, T=32768, E=256, k=8, S=16, score="softmax", half=False,
             masked=False, padded=False),
    ]


def _size(rng, lo, hi, unit=1):
    """A multiple of `unit`, spread over the logarithm."""
    return unit * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "balance"])
    if op == "norm":
        H = _size(rng, 8, 1024, 8)
        fp8 = rng.random() < 0.3 and H % 16 == 0
        branch = rng.random() < 0.8
        return dict(op="norm", T=max(1, min(_size(rng, 1, 16384), (8192 * 4096) // H)), H=H,
                    kind=rng.choice(["rms", "rms", "layer"]), stream32=rng.random() < 0.5, branch=branch,
                    post=branch and rng.random() < 0.4,
                    gate=rng.choice(["none", "none", "token", "channel", "element"]) if branch else "none",
                    half=not fp8 or rng.random() < 0.5, fp8=fp8, offset=rng.choice([0.0, 0.0, 1.0]))
    if op == "linear":
        K, N = _size(rng, 8, 1024, 8), _size(rng, 8, 8192)
        T = max(1, min(_size(rng, 1, 8192), (8192 * 8192 * 4096) // (N * K)))
        return dict(op="linear", T=T, N=N, K=K,
                    act=rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid"]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5, out32=rng.random() < 0.4)
    E = _size(rng, 4, 1024)
    T = max(1, min(_size(rng, 1, 32768), (32768 * 256) // E))
    return dict(op="balance", back=rng.random() < 0.5, T=T, E=E, k=rng.randint(1, min(16, E)), S=_size(rng, 1, 32),
                score=rng.choice(["softmax", "sigmoid"]), half=rng.random() < 0.3, masked=rng.random() < 0.25,
                padded=rng.random() < 0.3)


def work(case):
    c = case
    if c["op"] == "norm":
        n, s = c["T"] * c["H"], 4 if c["stream32"] else 2
        read = n * s + 2 * c["H"]
        if c["branch"]:  # the branch, and the stream written back
            read += n * (2 + s) + (2 * c["H"] if c["post"] else 0)
            read += {"none": 0, "token": 4 * c["T"], "channel": 2 * c["H"], "element": 2 * n}[c["gate"]]
        return {"bytes": read + (2 * n if c["half"] else 0) + (n + 4 * c["T"] * -(-c["H"] // 128) if c["fp8"] else 0),
                "flops": 12 * n}
    if c["op"] == "linear":
        T, N, K, e = c["T"], c["N"], c["K"], 4 if c["out32"] else 2
        return {"bytes": 2 * (T + N) * K + (4 * N if c["bias"] else 0) + (2 if c["residual"] else 1) * e * T * N,
                "flops": 2 * T * N * K}
    T, E, e = c["T"], c["E"], 2 if c["half"] else 4
    table = 4 * c["S"] * (E + 2)
    if c["back"]:
        return {"bytes": T * E * (e + 4) + table, "flops": 8 * T * E}
    return {"bytes": T * E * e + 4 * T * c["k"] + table + 4 * c["S"] * E, "flops": 6 * T * E}


# ---- inputs -----------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]
    typ = torch.float32 if c["stream32"] else torch.float16
    # A residual stream: some channels much larger than the others.
    x = _randn(g, T, H) * torch.where(torch.rand((H,), generator=g, device=DEV) < 0.01, 20.0, 1.5)
    layer = c["kind"] == "layer"
    vec = lambda: (1.0 - c["offset"] + 0.2 * _randn(g, H)).half()  # noqa: E731
    st = dict(c=c, x=x.to(typ), w=vec(), b=(0.1 * _randn(g, H)).half() if layer else None, branch=None, pw=None,
              pb=None, gate=None, scale=1.0, rscale=1.0)
    if c["branch"]:
        st["branch"] = (0.7 * _randn(g, T, H)).half()
        st["scale"], st["rscale"] = 0.75, 1.25
        if c["post"]:
            st["pw"], st["pb"] = vec(), (0.1 * _randn(g, H)).half() if layer else None
        if c["gate"] == "token":
            st["gate"] = torch.rand((T,), generator=g, device=DEV)
        elif c["gate"] == "channel":
            st["gate"] = (0.5 + 0.2 * _randn(g, H)).half()
        elif c["gate"] == "element":
            st["gate"] = (0.5 + 0.2 * _randn(g, T, H)).half()
    new = lambda *s, d: torch.empty(s, dtype=d, device=DEV)  # noqa: E731
    st["h"] = new(T, H, d=typ) if c["branch"] else None
    st["y"] = new(T, H, d=torch.float16) if c["half"] else None
    st["q"] = new(T, H, d=torch.float8_e4m3fn) if c["fp8"] else None
    st["s"] = new(T, -(-H // 128), d=torch.float32) if c["fp8"] else None
    if own:  # the norm's settings, made once per model
        st["cfg"] = _moe().moe_norm_config(kind=c["kind"], eps=1e-6, weight_offset=c["offset"])
    return st


def _prepare_linear(c, g):
    T, N, K = c["T"], c["N"], c["K"]
    typ = torch.float32 if c["out32"] else torch.float16
    x = _randn(g, T, K) * torch.where(torch.rand((K,), generator=g, device=DEV) < 0.01, 12.0, 1.0)
    w = _randn(g, N, K) * (1.2 / math.sqrt(K)) * torch.exp(0.2 * _randn(g, N, 1))
    st = dict(c=c, x=x.half(), w=w.half(), b=0.5 * _randn(g, N) if c["bias"] else None,
              r=_randn(g, T, N).to(typ) if c["residual"] else None, y=torch.empty((T, N), dtype=typ, device=DEV))
    if own:  # the workspace that a program keeps
        st["work"] = torch.zeros(_moe().moe_linear_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    return st


def _prepare_balance(c, g):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    l = 1.5 * _randn(g, T, E) + 0.5 * _randn(g, E)
    if c["half"]:
        l = l.half()
    if c["masked"]:
        l = l.masked_fill(torch.rand((T, E), generator=g, device=DEV) < 0.3, -math.inf)
        l[T // 2::97] = -math.inf  # tokens whose mask leaves no expert
    value, ids = l.float().topk(k, dim=1)
    ids = torch.where(value > -math.inf, ids, -1).int()
    # Sequences end to end, of ragged lengths; one of them empty; behind them, perhaps, padding.
    cuts = torch.rand((S + 1,), generator=g, device=DEV).sort()[0]
    ends = (cuts * (T + 1)).floor().int().clamp(max=T)
    ends[0] = 0
    if not c["padded"]:
        ends[S] = T
    if S > 2:
        ends[S // 2] = ends[S // 2 - 1]
    st = dict(c=c, logits=l, ids=ids, offsets=ends, coef=0.01, grad=torch.rand((1,), generator=g, device=DEV) + 0.5)
    if own:  # the loss's settings and buffers, kept by a training loop
        st["cfg"] = _moe().moe_balance_config(score=c["score"], coef=st["coef"])
        st["counts"] = torch.empty((S, E), dtype=torch.int32, device=DEV)
        st["tokens"] = torch.empty((S,), dtype=torch.int32, device=DEV)
        st["mean"] = torch.empty((S, E), dtype=torch.float32, device=DEV)
        st["loss"] = torch.empty((1,), dtype=torch.float32, device=DEV)
        st["work"] = torch.zeros(_moe().moe_balance_workspace_bytes(T, E, S), dtype=torch.uint8, device=DEV)
        st["dlogits"] = torch.zeros((T, E), dtype=torch.float32, device=DEV)
    if c["back"]:  # what the forward pass left
        st["fc"], st["fn"] = _counts(c, l, ids, ends)
    return st


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    return {"norm": _prepare_norm, "linear": _prepare_linear, "balance": _prepare_balance}[c["op"]](c, g)


# ---- plain forms --------------------------------------------------------------
def _moe():
    from int4_routed_expert_moe_gb300 import moe
    return moe


def _norm(c, v, w, b):
    if c["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * (w.float() + c["offset"])
    return v if b is None else v + b.float()


def _quantize(v):
    """E4M3 codes and FP32 scales of blocks of 1 x 128: s = amax / 448, q = v * (448 / amax)."""
    T, H = v.shape
    nb = -(-H // 128)
    p = torch.nn.functional.pad(v, (0, 128 * nb - H)).view(T, nb, 128)
    amax = p.abs().amax(2)
    q = (p * torch.where(amax > 0, E4M3_MAX / amax, 0.0)[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(T, 128 * nb)[:, :H].contiguous(), amax / E4M3_MAX


def _plain_norm(st):
    c, h, out = st["c"], st["x"].float(), {}
    if c["branch"]:
        a = st["branch"].float()
        if c["post"]:
            a = _norm(c, a, st["pw"], st["pb"])
        if st["gate"] is not None:
            a = a * (st["gate"].float()[:, None] if c["gate"] == "token" else st["gate"].float())
        h = st["rscale"] * h + st["scale"] * a
        out["h"] = h.to(st["x"].dtype)
    y = _norm(c, h, st["w"], st["b"])
    if c["half"]:
        out["y"] = y.half()
    if c["fp8"]:
        out["q"], out["scales"] = _quantize(y)
    return out


def _act(name, v):
    if name == "relu":
        return torch.where(v > 0, v, 0.0 * v)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    return v


def _plain_linear(st):
    c, v = st["c"], st["x"].float() @ st["w"].float().t()
    if st["b"] is not None:
        v = v + st["b"]
    v = _act(c["act"], v)
    if st["r"] is not None:
        v = v + st["r"].float()
    return v.to(st["y"].dtype)


def _members(c, l, offsets):
    """[S][T]: which tokens each sequence has (64 bits: their long sums are products with it), and which of them count."""
    t = torch.arange(c["T"], device=l.device)
    inside = (t >= offsets[:-1, None]) & (t < offsets[1:, None])
    good = (l > -math.inf).any(1) & ~(torch.isnan(l) | (l == math.inf)).any(1)
    return inside, inside & good


def _counts(c, l, ids, offsets):
    inside, valid = _members(c, l, offsets)
    picked = torch.zeros((c["T"], c["E"] + 1), dtype=torch.float64, device=l.device)
    picked.scatter_(1, torch.where(ids < 0, c["E"], ids).long(), 1.0)  # a token's picks differ
    return (inside.double() @ picked[:, :c["E"]]).int(), valid.sum(1).int()


def _probs(c, l):
    """The router's probabilities, and sigmoid(l); bad tokens' are zero. Their sums are taken in 64 bits."""
    l = l.float()
    if c["score"] == "softmax":
        s = None
        p = torch.exp(l - l.max(1, keepdim=True)[0])
    else:
        p = s = 1.0 / (1.0 + torch.exp(-l))
    return p / p.sum(1, keepdim=True), s


def _plain_balance(st):
    c, l, E = st["c"], st["logits"], st["c"]["E"]
    inside, valid = _members(c, l, st["offsets"])
    p, s = _probs(c, l)
    p = torch.where(valid.any(0)[:, None], p, 0.0)
    if not c["back"]:
        counts, n = _counts(c, l, st["ids"], st["offsets"])
        each = n.clamp(min=1).double()[:, None]
        mean = (valid.double() @ p.double()) / each
        f = counts.double() * (E / c["k"]) / each
        live = (n > 0).sum().clamp(min=1)
        loss = st["coef"] * ((f * mean) * (n > 0)[:, None]).sum() / live
        return {"loss": loss.float().reshape(1), "counts": counts, "tokens": n, "mean": mean.float()}
    n = st["fn"].clamp(min=1).double()[:, None]
    live = (st["fn"] > 0).sum().clamp(min=1)
    f = st["fc"].double() * (E / c["k"]) / n * (st["coef"] * st["grad"].double() / live / n)
    f = f[valid.int().argmax(0)].float()  # each token's sequence
    d = p * (f - (f * p).sum(1, keepdim=True))
    if s is not None:
        d = d * (1.0 - s)
    return {"dlogits": torch.where(valid.any(0)[:, None], d, 0.0)}


def run(state):
    st, c = state, state["c"]
    if c["op"] == "norm":
        if not own:
            return _plain_norm(st)
        if c["branch"]:
            _moe().moe_norm_residual(st["cfg"], st["branch"], st["x"], st["h"], st["pw"], st["pb"], st["gate"],
                                     st["scale"], st["rscale"], st["w"], st["b"], st["y"], st["q"], st["s"])
        else:
            _moe().moe_norm(st["cfg"], st["x"], st["w"], st["b"], st["y"], st["q"], st["s"])
        out = {"h": st["h"], "y": st["y"], "q": st["q"], "scales": st["s"]}
        return {n: t for n, t in out.items() if t is not None}
    if c["op"] == "linear":
        if not own:
            return _plain_linear(st)
        _moe().moe_linear(st["x"], st["w"], st["b"], st["y"], st["work"], c["act"], st["r"])
        return st["y"]
    if not own:
        return _plain_balance(st)
    if c["back"]:
        _moe().moe_balance_loss_backward(st["cfg"], st["logits"], c["k"], st["offsets"], st["fc"], st["fn"], st["grad"],
                                         st["dlogits"])
        return {"dlogits": st["dlogits"]}
    _moe().moe_balance_loss(st["cfg"], st["logits"], st["ids"], st["offsets"], st["counts"], st["tokens"], st["mean"],
                            st["loss"], st["work"])
    return {"loss": st["loss"], "counts": st["counts"], "tokens": st["tokens"], "mean": st["mean"]}


# ---- 64 bits ------------------------------------------------------------------
def _exact_norm_row(c, v, w, b):
    w = w.double() + c["offset"]
    if c["kind"] == "layer":
        var, mu = torch.var_mean(v, dim=1, unbiased=False, keepdim=True)
        v = v - mu
    else:
        var = torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / v.shape[1]
    v = w * v * (var + 1e-6) ** -0.5
    return v + b.double() if b is not None else v


def _exact_codes(v):
    """Nearest E4M3 value of each |v| <= 448, ties to even: 3 bits after the leading one, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(st):
    c, out = st["c"], {}
    h = st["x"].double()
    if c["branch"]:
        a = st["branch"].double()
        if c["post"]:
            a = _exact_norm_row(c, a, st["pw"], st["pb"])
        if c["gate"] == "token":
            a = a * st["gate"].double().unsqueeze(1)
        elif c["gate"] != "none":
            a = a * st["gate"].double()
        h = h * st["rscale"] + a * st["scale"]
        out["h"] = h
    y = _exact_norm_row(c, h, st["w"], st["b"])
    if c["half"]:
        out["y"] = y
    if c["fp8"]:
        cols = [y[:, i:i + 128] for i in range(0, c["H"], 128)]
        top = [t.abs().max(1, keepdim=True)[0] for t in cols]
        out["q"] = torch.cat([_exact_codes(torch.where(m > 0, t * E4M3_MAX / m, 0.0)) for t, m in zip(cols, top)], 1)
        out["scales"] = torch.cat(top, 1) / E4M3_MAX
    return out


def _exact_linear(st):
    c = st["c"]
    w, rows = st["w"].double().t().contiguous(), []
    for x in st["x"].split(2048):
        v = x.double() @ w
        if c["bias"]:
            v += st["b"].double()
        if c["act"] == "relu":
            v = v.clamp(min=0.0)
        elif c["act"] in ("silu", "sigmoid"):
            g = torch.special.expit(v)
            v = g * v if c["act"] == "silu" else g
        elif c["act"] == "gelu":
            v = v * torch.special.ndtr(v)
        elif c["act"] == "gelu_tanh":
            v = v * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
        rows.append(v)
    y = torch.cat(rows)
    return y + st["r"].double() if c["residual"] else y


def _exact_balance(st):
    """Sequence by sequence, on the host."""
    c, E, k = st["c"], st["c"]["E"], st["c"]["k"]
    l, ids = st["logits"].cpu().numpy().astype(np.float64), st["ids"].cpu().numpy()
    off = st["offsets"].cpu().numpy()
    S, T = c["S"], c["T"]
    counts, n, mean = np.zeros((S, E), np.int32), np.zeros(S, np.int32), np.zeros((S, E))
    d = np.zeros((T, E))
    alive = []
    for s in range(S):
        a, b = int(off[s]), int(off[s + 1])
        i = ids[a:b]
        counts[s] = np.bincount(i[i >= 0], minlength=E)
        good = np.flatnonzero(np.isfinite(l[a:b]).any(1)) + a
        n[s] = len(good)
        if len(good):
            x = l[good]
            sig = 1.0 / (1.0 + np.exp(-x))
            e = sig if c["score"] == "sigmoid" else np.exp(x - x.max(1)[:, None])
            p = e / e.sum(1)[:, None]
            mean[s] = p.mean(0)
            alive.append((s, good, p, 1.0 - sig if c["score"] == "sigmoid" else np.ones_like(p)))
    share = st["coef"] / max(1, len(alive))
    if not c["back"]:
        loss = sum(share * E * float(counts[s] @ mean[s]) / (k * int(n[s])) for s, _, _, _ in alive)
        return {"loss": np.array([loss]), "counts": counts, "tokens": n, "mean": mean}
    grad = float(st["grad"].double())
    for s, good, p, outer in alive:
        f = counts[s] * (E / (k * float(n[s])))
        d[good] = grad * share / float(n[s]) * p * (f[None, :] - (p @ f)[:, None]) * outer
    return {"dlogits": d}


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "balance": _exact_balance}[case["op"]](st)
