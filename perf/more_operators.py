"""A gated linear recurrence, a gated feed-forward block and the log probabilities of tokens: cases,
inputs, plain forms, exact values.

``run`` computes the plain forms from elementary torch operations, in 32 bits whatever the
inputs' type and rounded once at the end; with ``own`` set it makes the framework's calls.

Operators (``case["op"]``):

* ``lru``: the gated linear recurrence over [batch, dim, seqlen]: r = sigmoid(gate_a),
  i = sigmoid(gate_x), a = exp(lam r), h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t.  "fwd" is the
  forward with a carried state, "train" a forward and the backward that follows it.
* ``logprob``: rows of logits: the log probability of a given token per row, the logarithm of the
  sum, the entropy and the `top` likeliest tokens ("fwd"), or the gradient of those ("bwd").
* ``mlp``: act(x Wg^T) * (x Wu^T) ("fwd"), or its gradients ("bwd").
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ---- cases ------------------------------------------------------------------------------------

def _lru(mode, batch, dim, seqlen, dtype, carried=True):
    return dict(op="lru", mode=mode, batch=batch, dim=dim, seqlen=seqlen, dtype=dtype,
                carried=carried)


def _logprob(mode, rows, vocab, dtype, top=0, entropy=True, scale=1.0, masked=False,
             long_ids=True):
    return dict(op="logprob", mode=mode, rows=rows, vocab=vocab, dtype=dtype, top=top,
                entropy=entropy, scale=scale, masked=masked, long_ids=long_ids)


def _mlp(mode, tokens, dim, hidden, dtype, act="silu"):
    return dict(op="mlp", mode=mode, tokens=tokens, dim=dim, hidden=hidden, dtype=dtype, act=act)


def listed():
    cases = [
        # 64 sequences decoded together, one token each: the call's latency
        ("lru_fwd_decode", _lru("fwd", 64, 1536, 1, "bf16")),
        # one long sequence of a wide model, from a state carried into it
        ("lru_fwd_long", _lru("fwd", 1, 5120, 65536, "bf16")),
        # the mixer of a training step, 8 x 2048 tokens of 1536 channels
        ("lru_train", _lru("train", 8, 1536, 2048, "bf16", carried=False)),
        # few channels over a long odd sequence in fp32: the work has to be split over time
        ("lru_train_few", _lru("train", 2, 100, 30011, "f32")),
        # scoring a training batch: 8 x 2048 tokens of a vocabulary of 50257
        ("logprob_fwd_train", _logprob("fwd", 16384, 50257, "bf16")),
        # the gradient of the loss on that batch
        ("logprob_bwd_train", _logprob("bwd", 16384, 50257, "bf16", entropy=False)),
        # 64 sequences decoded together: masked logits, entropy and 20 alternatives
        ("logprob_fwd_decode", _logprob("fwd", 64, 50257, "f32", top=20, masked=True)),
        # the selective-copying task: 64 x 4096 tokens of a vocabulary of 16
        ("logprob_bwd_copying", _logprob("bwd", 262144, 16, "f32", long_ids=False)),
        # 8 sequences decoded together: every weight is read for them
        ("mlp_fwd_decode", _mlp("fwd", 8, 2048, 5632, "bf16")),
        # a training batch of 8 x 2048 tokens in a wider model
        ("mlp_fwd_train", _mlp("fwd", 16384, 2048, 5632, "bf16")),
        # the backward of a training step, 8 x 2048 tokens of width 768
        ("mlp_bwd_train", _mlp("bwd", 16384, 768, 2048, "bf16")),
        # sizes that no tile divides, in fp32, with the other activation
        ("mlp_bwd_odd", _mlp("bwd", 777, 1000, 2603, "f32", "gelu")),
    ]
    return [dict(case, name=name) for name, case in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: mostly a multiple of 64 or 8, else any."""
    n = _log(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(("lru", "logprob", "mlp"))
    dtype = rng.choice(("f32", "bf16", "bf16"))
    if op == "lru":
        dim = _width(rng, 16, 8192)
        batch = _log(rng, 1, 64)
        seqlen = _log(rng, 1, max(1, min(65536, (1 << 25) // (dim * batch))))
        return _lru(rng.choice(("fwd", "train")), batch, dim, seqlen, dtype, rng.random() < 0.5)
    if op == "logprob":
        vocab = rng.choice((_width(rng, 2, 1024), _width(rng, 1024, 160000)))
        mode = rng.choice(("fwd", "bwd"))
        top = rng.choice((0, 0, 1, 5, 20, 64)) if mode == "fwd" else 0
        rows = _log(rng, 1, max(2, min(65536 if top == 0 else 2048, (1 << 27) // vocab)))
        return _logprob(mode, rows, vocab, dtype, min(top, vocab), rng.random() < 0.6,
                        rng.choice((1.0, 1.0, 0.7, 1.6)), rng.random() < 0.4, rng.random() < 0.7)
    dim, hidden = _width(rng, 32, 4096), _width(rng, 32, 8192)
    most = (1 << 35) if dtype == "bf16" else (1 << 33)
    tokens = _log(rng, 1, max(2, min(16384, most // (dim * hidden))))
    return _mlp(rng.choice(("fwd", "bwd")), tokens, dim, hidden, dtype,
                rng.choice(("silu", "silu", "gelu")))


def work(case):
    t = BYTES[case["dtype"]]
    if case["op"] == "lru":
        rows = case["batch"] * case["dim"]
        n = rows * case["seqlen"]
        state = 4 * rows * (2 if case["carried"] else 1) + 4 * case["dim"]
        if case["mode"] == "fwd":  # x and two gates in, out
            return {"bytes": 4 * n * t + state, "flops": 20 * n}
        # and for the backward x, two gates and dout in, three gradients out
        return {"bytes": 11 * n * t + state + 4 * case["dim"], "flops": 60 * n}
    if case["op"] == "logprob":
        n, r = case["rows"] * case["vocab"], case["rows"]
        ids = r * (8 if case["long_ids"] else 4)
        if case["mode"] == "fwd":
            per = 8 + (4 if case["entropy"] else 0) + 12 * case["top"]
            return {"bytes": n * t + ids + r * per, "flops": 6 * n}
        return {"bytes": 2 * n * t + ids + r * (12 if case["entropy"] else 8), "flops": 6 * n}
    m, d, f = case["tokens"], case["dim"], case["hidden"]
    if case["mode"] == "fwd":
        return {"bytes": t * (m * d + 2 * f * d + m * f), "flops": 4 * m * f * d}
    # the two projections again, the gradient of x, the gradients of the weights
    return {"bytes": t * (2 * m * d + 4 * f * d + m * f), "flops": 12 * m * f * d}


# ---- inputs -----------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        x = torch.empty(shape, device="cuda", dtype=DTYPES[dtype])
        return x.normal_(mean, std, generator=g)

    st = dict(case)
    if case["op"] == "lru":
        shape = (case["batch"], case["dim"], case["seqlen"])
        for k in ("x", "gate_a", "gate_x"):
            st[k] = normal(shape, case["dtype"], 1.0 if k == "x" else 1.5)
        # a^2 at an open gate between 0.9^2 and 0.999^2, its rate eight times that of the gate
        u = torch.rand((case["dim"],), device="cuda", generator=g) * 0.099 + 0.9
        st["lam"] = 8.0 * torch.log(u)
        st["h0"] = normal(shape[:2], "f32") if case["carried"] else None
        if case["mode"] == "train":
            st["dout"] = normal(shape, case["dtype"])
    elif case["op"] == "logprob":
        r, v = case["rows"], case["vocab"]
        st["logits"] = normal((r, v), case["dtype"], 2.5)
        if case["masked"]:  # tokens that may not follow
            off = torch.rand((r, v), device="cuda", generator=g) < 0.3
            st["logits"][off] = -math.inf
        ids = torch.randint(v, (r,), device="cuda", generator=g)
        pad = torch.rand((r,), device="cuda", generator=g) < 0.05  # padding: no token asked for
        ids = torch.where(pad, -100, ids)
        st["ids"] = ids if case["long_ids"] else ids.int()
        if case["mode"] == "bwd":
            st["dlogprob"] = normal((r,), "f32", 1.0 / r, -1.0 / r)
            # what the forward left
            s = torch.full((r,), -math.inf, device="cuda", dtype=torch.float64)
            e = torch.zeros((r,), device="cuda", dtype=torch.float64)
            step = max(1, (1 << 26) // v)
            for a in range(0, r, step):
                x = st["logits"][a:a + step].double() * case["scale"]
                s[a:a + step] = torch.logsumexp(x, -1)
                p = torch.exp(x - s[a:a + step, None])
                e[a:a + step] = s[a:a + step] - torch.where(p > 0, p * x, 0.0).sum(-1)
            st["lse"] = s.float()
            e = torch.where(torch.isinf(s), 0.0, e)  # nothing is left in such a row
            st["entropy_of"] = e.float() if case["entropy"] else None
            st["dentropy"] = normal((r,), "f32", 0.1 / r) if case["entropy"] else None
    else:
        m, d, f = case["tokens"], case["dim"], case["hidden"]
        st["x"] = normal((m, d), case["dtype"])
        st["w_gate"] = normal((f, d), case["dtype"], 1.0 / math.sqrt(d))
        st["w_up"] = normal((f, d), case["dtype"], 1.0 / math.sqrt(d))
        if case["mode"] == "bwd":
            st["dout"] = normal((m, f), case["dtype"])
    return st


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import selective_state_space_26_amd as msel
    if st["op"] == "lru":
        a = (st["x"], st["gate_a"], st["gate_x"], st["lam"])
        if st["mode"] == "fwd":
            return list(msel.msel_lru_fwd(*a, st["h0"])[:2])
        out, final, chunks = msel.msel_lru_fwd(*a, st["h0"], return_chunk_states=True)
        r = msel.msel_lru_bwd(*a, st["dout"], st["h0"], chunk_states=chunks,
                              want_dh0=st["carried"])
        return [out, final, r["dx"], r["dgate_a"], r["dgate_x"], r["dlam"], r["dh0"]]
    if st["op"] == "logprob":
        if st["mode"] == "fwd":
            r = msel.msel_logprob_fwd(st["logits"], st["ids"], st["scale"], st["top"],
                                      want_entropy=st["entropy"])
            return [r["logprob"], r["lse"], r["entropy"], r["top_ids"], r["top_logprobs"]]
        return msel.msel_logprob_bwd(st["logits"], st["ids"], st["lse"], st["dlogprob"],
                                     dentropy=st["dentropy"], entropy=st["entropy_of"],
                                     scale=st["scale"])
    a = (st["x"], st["w_gate"], st["w_up"])
    if st["mode"] == "fwd":
        return msel.msel_gated_mlp_fwd(*a, st["act"])
    r = msel.msel_gated_mlp_bwd(*a, st["dout"], st["act"])
    return [r["dx"], r["dw_gate"], r["dw_up"]]


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the last axis from 0, by doubling spans of composed steps."""
    n, s = a.shape[-1], 1
    while s < n:
        b = torch.cat([b[..., :s], b[..., s:] + a[..., s:] * b[..., :-s]], -1)
        if 2 * s < n:
            a = torch.cat([a[..., :s], a[..., s:] * a[..., :-s]], -1)
        s *= 2
    return b


def _lru_plain(st):
    act = DTYPES[st["dtype"]]
    x, lam = st["x"].float(), st["lam"][:, None]
    r, i = _sigmoid(st["gate_a"].float()), _sigmoid(st["gate_x"].float())
    la = lam * r
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2.0 * la))
    b = m * i * x
    if st["h0"] is not None:
        b[..., 0] += a[..., 0] * st["h0"]
    h = _scan(a, b)
    out = [h.to(act), h[..., -1].clone()]
    if st["mode"] == "fwd":
        return out
    before = torch.zeros_like(h[..., 0]) if st["h0"] is None else st["h0"]
    before = torch.cat([before[..., None], h[..., :-1]], -1)
    # the adjoint runs backwards: g_t = dout_t + a_{t+1} g_{t+1}
    after = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], -1)
    g = _scan(after.flip(-1), st["dout"].float().flip(-1)).flip(-1)
    dla = g * (a * before - torch.where(m > 0, i * x * a * a / m, 0.0))
    return out + [(g * m * i).to(act), (dla * lam * r * (1.0 - r)).to(act),
                  (g * m * x * i * (1.0 - i)).to(act), (dla * r).sum((0, 2)),
                  a[..., 0] * g[..., 0] if st["carried"] else None]


def _logprob_plain(st):
    """A row whose tokens are all masked has probabilities of 0, no entropy and no gradient."""
    x = st["logits"].float() * st["scale"]
    ids = st["ids"].long()
    real = (ids >= 0) & (ids < st["vocab"])
    at = torch.where(real, ids, 0)[:, None]
    if st["mode"] == "fwd":
        top = x.max(-1, keepdim=True).values
        top = torch.where(torch.isinf(top), 0.0, top)
        e = torch.exp(x - top)
        s = e.sum(-1, keepdim=True)
        lse = top + torch.log(s)
        lp = torch.where(s > 0, x.gather(1, at) - lse, -math.inf)
        out = [torch.where(real, lp[:, 0], 0.0), lse[:, 0], None, None, None]
        if st["entropy"]:
            spread = torch.where(e > 0, e * (x - top), 0.0).sum(-1, keepdim=True)
            out[2] = torch.where(s > 0, torch.log(s) - spread / s, 0.0)[:, 0]
        if st["top"]:
            ids = torch.sort(st["logits"].float(), dim=-1, descending=True, stable=True).indices
            out[3] = ids[:, :st["top"]].contiguous()
            out[4] = torch.where(s > 0, x.gather(1, out[3]) - lse, -math.inf)
        return out
    lp = x - st["lse"][:, None]
    p = torch.exp(lp)
    dlp = torch.where(real, st["dlogprob"], 0.0)[:, None]
    d = -p * dlp
    d.scatter_add_(1, at, dlp)
    if st["entropy"]:
        h = st["dentropy"][:, None] * (lp + st["entropy_of"][:, None])
        d -= torch.where(p > 0, p * h, 0.0)
    d = torch.where(torch.isinf(st["lse"])[:, None], 0.0, d * st["scale"])
    return d.to(st["logits"].dtype)


ROOT_2_PI = math.sqrt(2.0 / math.pi)


def _act_and_slope(z, act):
    if act == "silu":
        s = _sigmoid(z)
        return z * s, s * (1.0 + z * (1.0 - s))
    t = torch.tanh(ROOT_2_PI * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * ROOT_2_PI
                                 * (1.0 + 3 * 0.044715 * z * z))


def _mlp_plain(st):
    act = DTYPES[st["dtype"]]
    x, wg, wu = (st[k].float() for k in ("x", "w_gate", "w_up"))
    v, slope = _act_and_slope(x @ wg.T, st["act"])
    u = x @ wu.T
    if st["mode"] == "fwd":
        return (v * u).to(act)
    dout = st["dout"].float()
    dg, du = dout * u * slope, dout * v
    return [(dg @ wg + du @ wu).to(act), (dg.T @ x).to(act), (du.T @ x).to(act)]


def _run_plain(st):
    return {"lru": _lru_plain, "logprob": _logprob_plain, "mlp": _mlp_plain}[st["op"]](st)


# ---- the definition in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"lru": _lru_exact, "logprob": _logprob_exact, "mlp": _mlp_exact}[case["op"]](st)


def _lru_exact(st):
    """Step by step over time, channels of all sequences together."""
    L = st["seqlen"]
    by_time = lambda t: t.permute(2, 0, 1).double().contiguous()  # noqa: E731
    r, i = torch.sigmoid(by_time(st["gate_a"])), torch.sigmoid(by_time(st["gate_x"]))
    la = r * st["lam"].double()
    a, m = la.exp(), (-torch.expm1(2 * la)).sqrt()
    x = by_time(st["x"])
    b = m * i * x
    h = torch.zeros_like(x[0]) if st["h0"] is None else st["h0"].double()
    hs = torch.empty((L + 1,) + h.shape, device="cuda", dtype=torch.float64)
    hs[0] = h
    for t in range(L):
        torch.addcmul(b[t], a[t], hs[t], out=hs[t + 1])
    back = lambda t: t.permute(1, 2, 0)  # noqa: E731
    out = [back(hs[1:]), hs[L]]
    if st["mode"] == "fwd":
        return out
    d = by_time(st["dout"])
    for t in range(L - 2, -1, -1):  # d becomes the adjoint
        d[t].addcmul_(a[t + 1], d[t + 1])
    root = torch.where(m > 0, a * a * i * x / m, torch.zeros_like(m))
    dla = d * (a * hs[:-1] - root)
    return out + [back(d * m * i), back(dla * st["lam"].double() * r * (1 - r)),
                  back(d * m * x * i * (1 - i)), (dla * r).sum((0, 1)),
                  a[0] * d[0] if st["carried"] else None]


def _logprob_exact(st):
    rows, v = st["rows"], st["vocab"]
    step = max(1, (1 << 26) // v)
    parts = []
    for n in range(0, rows, step):
        x = st["logits"][n:n + step].double() * st["scale"]
        ids = st["ids"][n:n + step].long()
        inside = (ids >= 0) & (ids < v)
        here = torch.arange(x.shape[0], device="cuda")[inside]
        some = (x > -math.inf).any(-1, keepdim=True)
        logp = torch.log_softmax(x, -1).masked_fill(~some, -math.inf)
        if st["mode"] == "fwd":
            lp = torch.zeros(x.shape[0], device="cuda", dtype=torch.float64)
            lp[inside] = logp[here, ids[inside]]
            one = [lp, torch.logsumexp(x, -1)]
            if st["entropy"]:
                one.append(torch.special.entr(logp.exp()).sum(-1))
            if st["top"]:
                order = torch.argsort(st["logits"][n:n + step].double(), dim=-1, descending=True,
                                      stable=True)[:, :st["top"]]
                one += [order, torch.take_along_dim(logp, order, 1)]
            parts.append(one)
            continue
        # d/dx of dlogprob log p_t + dentropy H with the forward's own sum and entropy
        p = torch.exp(x - st["lse"][n:n + step, None].double())
        w = torch.zeros(x.shape[0], device="cuda", dtype=torch.float64)
        w[inside] = st["dlogprob"][n:n + step].double()[inside]
        d = p * -w[:, None]
        d[here, ids[inside]] += w[inside]
        if st["entropy"]:
            h = st["entropy_of"][n:n + step].double()[:, None]
            d -= st["dentropy"][n:n + step].double()[:, None] * (
                -torch.special.entr(p) + p * h)
        parts.append([(d * st["scale"]).masked_fill(~some, 0.0)])
    out = [torch.cat(c) for c in zip(*parts)]
    if st["mode"] == "bwd":
        return out[0]
    full = out[:2] + [None, None, None]
    if st["entropy"]:
        full[2] = out[2]
    if st["top"]:
        full[3], full[4] = out[-2], out[-1]
    return full


def _mlp_exact(st):
    x, wg, wu = st["x"].double(), st["w_gate"].double(), st["w_up"].double()
    g, u = torch.nn.functional.linear(x, wg), torch.nn.functional.linear(x, wu)
    if st["act"] == "silu":
        s = torch.special.expit(g)
        value, slope = g * s, s + g * s * torch.special.expit(-g)
    else:
        inner = math.sqrt(2 / math.pi) * g * (1 + 0.044715 * g.square())
        s = torch.special.expit(2 * inner)  # (1 + tanh(inner)) / 2
        value = g * s
        slope = s + g * 2 * s * (1 - s) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g.square())
    if st["mode"] == "fwd":
        return value * u
    d = st["dout"].double()
    dg, du = d * u * slope, d * value
    return [torch.addmm(dg.mm(wg), du, wu), dg.t().mm(x), du.t().mm(x)]
