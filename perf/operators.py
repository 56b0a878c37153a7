"""Workloads of the recurrent block's operators: the gated linear recurrence
(sequence form, its backward, and the single-token step), the per-head norm
with its output gate (forward and backward), and the residual sum with the
norms around it (forward and backward).

`run` computes a case in its plain form (elementary torch operations in
float32, rounded once at the end) or, with `own` set, through the package.
`exact` evaluates the same definitions in float64, written apart from `run`.
"""
import math

import torch

own = False

CHUNK = 64    # tokens between two kept states of the recurrence
EPS = 1e-5


def listed():
    return [
        # One short float32 sequence, four heads of 64 channels: what a test or a small
        # model calls; its time is latency.
        dict(name="scan_tiny_f32", op="scan", B=1, N=256, D=256, dtype="f32", form="logit",
             gate=False, state=True, packed=False, train=False, fused=False),
        # Training forward of a 1.3B-class layer (batch 8, 2048 tokens, 8 heads of 256):
        # gate logits, input and output gate are slices of one projection.
        dict(name="scan_train_2k", op="scan", B=8, N=2048, D=2048, dtype="bf16", form="logit",
             gate=True, state=False, packed=False, train=True, fused=True),
        # Prefill of one long document at the 6.7B-class width: few channels, 65536 tokens,
        # log decays with resets where packed documents meet.
        dict(name="scan_prefill_64k", op="scan", B=1, N=65536, D=4096, dtype="bf16", form="log",
             gate=False, state=True, packed=True, train=False, fused=False),
        # Backward of the training forward above.
        dict(name="scan_backward_2k", op="scan_backward", B=8, N=2048, D=2048, dtype="bf16",
             form="logit", gate=True, state=False, packed=False, fused=True),
        # Backward at odd sizes in float32: a ragged tail in time and in channels.
        dict(name="scan_backward_odd_f32", op="scan_backward", B=3, N=1501, D=1001, dtype="f32",
             form="log", gate=False, state=True, packed=True, fused=False),
        # One decoded token at batch 8: latency.
        dict(name="scan_step_8", op="scan_step", B=8, D=4096, dtype="bf16", form="logit",
             gate=True, fused=True),
        # One decoded token of a large serving batch: the float32 states stream through.
        dict(name="scan_step_1024", op="scan_step", B=1024, D=8192, dtype="bf16", form="log",
             gate=False, fused=False),
        # Per-head GroupNorm and swish gate after retention, the 6.7B-class layer at 8k:
        # head-major in, token-major out for the output projection.
        dict(name="norm_gate_8k", op="norm_gate", B=8, H=16, N=8192, dv=512, dtype="bf16",
             norm="layer", gate=True, token_major=True),
        # Its backward in the 1.3B-class training layer.
        dict(name="norm_gate_backward_2k", op="norm_gate_backward", B=8, H=8, N=2048, dv=256,
             dtype="bf16", norm="layer", gate=True, token_major=True),
        # Residual and next norm of one decoded token at batch 8: latency.
        dict(name="add_norm_decode", op="add_norm", rows=8, d=4096, dtype="bf16", post="none",
             pre="rms", wpost=False, alpha=1.0, beta=1.0),
        # Both norms around the residual over a prefill of 8 x 2048 tokens, float32, odd width.
        dict(name="add_norm_odd_f32", op="add_norm", rows=16384, d=2001, dtype="f32",
             post="rms", pre="rms", wpost=True, alpha=1.0, beta=0.5),
        # Training backward of both norms, the 6.7B-class width over 8 x 8192 tokens.
        dict(name="add_norm_backward_64k", op="add_norm_backward", rows=65536, d=4096,
             dtype="bf16", post="rms", pre="layer", wpost=True, alpha=1.5, beta=0.7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width in [lo, hi]: a multiple of 64, a multiple of 8, or any number."""
    d = _log_int(rng, lo, hi)
    unit = rng.choice((64, 8, 1))
    return min(hi, max(lo, d // unit * unit))


def draw(rng):
    op = rng.choice(("scan", "scan_backward", "scan_step", "norm_gate", "norm_gate_backward",
                     "add_norm", "add_norm_backward"))
    c = dict(op=op, dtype=rng.choice(("bf16", "bf16", "f32")))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("scan", "scan_backward"):
        most = 1 << 26
        c["B"], c["D"] = rng.choice((1, 1, 2, 3, 5, 8)), _width(rng, 16, 8192)
        c["N"] = _log_int(rng, 1, max(1, min(65536, most // (c["B"] * c["D"]))))
        c |= dict(form=rng.choice(("logit", "log")), gate=flag(), state=flag(), packed=flag(),
                  fused=flag())
        if op == "scan":
            c["train"] = flag()
    elif op == "scan_step":
        c |= dict(B=_log_int(rng, 1, 1024), D=_width(rng, 16, 8192),
                  form=rng.choice(("logit", "log")), gate=flag(), fused=flag())
    elif op in ("norm_gate", "norm_gate_backward"):
        c |= dict(B=rng.choice((1, 2, 3, 8)), H=rng.choice((1, 3, 8, 16)),
                  dv=rng.choice((32, 40, 64, 96, 128, 256, 264, 512)))
        c["N"] = _log_int(rng, 1, min(65536, (1 << 26) // (c["B"] * c["H"] * c["dv"])))
        c |= dict(norm=rng.choice(("layer", "rms")), gate=rng.random() < 0.8, token_major=flag())
    else:
        c["d"] = _width(rng, 32, 8192)
        c["rows"] = _log_int(rng, 1, min(65536, (1 << 26) // c["d"]))
        c |= dict(post=rng.choice(("none", "rms", "layer")), pre=rng.choice(("rms", "layer")),
                  wpost=flag(), alpha=rng.choice((1.0, 1.5, 2.25)),
                  beta=rng.choice((1.0, 0.7, 0.25)))
    return c


# ---- what a program has in hand -------------------------------------------------

def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _forget(c, shape, normal, gen):
    """Gate logits or log decays with one time scale per channel (2 to 1000 tokens) and a
    spread from token to token."""
    tau = torch.exp(torch.rand(shape[-1], device="cuda", generator=gen) * math.log(500.0)
                    + math.log(2.0))
    if c["form"] == "logit":
        return torch.log(tau) + normal(shape)
    return -torch.nn.functional.softplus(normal(shape)) / tau


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(c)
    normal = lambda shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    s = dict(case=c)
    if c["op"] in ("scan", "scan_backward", "scan_step"):
        step = c["op"] == "scan_step"
        B, D = c["B"], c["D"]
        shape = (B, D) if step else (B, c["N"], D)
        if c["fused"]:  # x, f and the gate side by side, as one projection leaves them
            p = torch.empty(shape[:-1] + ((3 if c["gate"] else 2) * D,), device="cuda", dtype=dt)
            s["x"], s["f"] = p[..., :D], p[..., D:2 * D]
            g = p[..., 2 * D:] if c["gate"] else None
        else:
            s["x"], s["f"] = (torch.empty(shape, device="cuda", dtype=dt) for _ in range(2))
            g = torch.empty(shape, device="cuda", dtype=dt) if c["gate"] else None
        s["x"].copy_(normal(shape))
        s["f"].copy_(_forget(c, shape, normal, gen))
        if g is not None:
            g.copy_(normal(shape))
        s["gate"] = g
        if not step and c["packed"]:  # documents start here: nothing of the state before counts
            starts = torch.randint(0, c["N"], (max(1, c["N"] // 700),), device="cuda",
                                   generator=gen)
            s["f"][:, starts] = -math.inf
        if step:
            s["state"] = normal((B, D))
            s["new_state"] = torch.empty_like(s["state"])
        else:
            s["state"] = normal((B, D)) if c["state"] else None
        if c["op"] == "scan_backward":
            s["d_y"] = normal(shape).to(dt)
            s["d_state"] = normal((B, D)) if c["state"] else None
            s["chunk_states"] = _kept(_hidden(s)[0], s["state"])
    elif c["op"] in ("norm_gate", "norm_gate_backward"):
        B, H, N, dv = c["B"], c["H"], c["N"], c["dv"]
        out = (B, N, H, dv) if c["token_major"] else (B, H, N, dv)
        # retention outputs: rows of very different lengths, not centred
        s["y"] = (normal((B, H, N, dv)) * torch.exp(normal((B, H, N, 1)))
                  + 0.3 * normal((B, H, N, 1))).to(dt)
        s["gate"] = normal(out).to(dt) if c["gate"] else None
        if c["op"] == "norm_gate_backward":
            s["d_o"] = normal(out).to(dt)
    else:
        rows, d = c["rows"], c["d"]
        s["x"] = normal((rows, d)).to(dt)
        s["w_pre"] = 1 + 0.2 * normal((d,))
        s["w_post"] = 1 + 0.2 * normal((d,)) if c["wpost"] else None
        # the residual stream: a few channels much larger than the rest
        r = normal((rows, d)) * (1 + 8 * (torch.rand(d, device="cuda", generator=gen) < 0.02))
        s["residual"] = r.to(dt)
        if c["op"] == "add_norm_backward":
            s["d_y"] = normal((rows, d)).to(dt)
            s["d_res"] = normal((rows, d)).to(dt)
    return s


# ---- plain forms, float32 ----------------------------------------------------------

def _gates(f, form):
    """The decay a and 1 - a, float32.  A log decay lies close under 0 and its power close
    under 1, where a last-bit error repeats over hundreds of tokens: taken in float64."""
    if form == "logit":
        f = f.float()
        return torch.sigmoid(f), torch.sigmoid(-f)
    return torch.exp(f.double()).float(), -torch.expm1(f.float())


def _recur(a, u):
    """h_t = a_t h_(t-1) + u_t over dim 1, by doubling: after each round h_t holds the
    terms of twice as many tokens (log2 N rounds)."""
    a, h, reach = a.clone(), u.clone(), 1
    while reach < a.shape[1]:
        h[:, reach:] = h[:, reach:] + a[:, reach:] * h[:, :-reach]
        a[:, reach:] = a[:, reach:] * a[:, :-reach]
        reach *= 2
    return h


def _hidden(s):
    a, rest = _gates(s["f"], s["case"]["form"])
    u = s["x"].float()
    u = rest * u if s["case"]["form"] == "logit" else u.clone()
    if s["state"] is not None:
        u[:, 0] += a[:, 0] * s["state"]
    return _recur(a, u), a, rest


def _kept(h, state):
    """The state entering every CHUNK tokens, [B, chunks, D]."""
    first = torch.zeros_like(h[:, :1]) if state is None else state[:, None]
    return torch.cat([first, h[:, CHUNK - 1:h.shape[1] - 1:CHUNK]], 1)


def _swish(g):
    g = g.float()
    return g * torch.sigmoid(g)


def _scan(s):
    h, _, _ = _hidden(s)
    y = h if s["gate"] is None else h * _swish(s["gate"])
    out = {"y": y.to(s["x"].dtype), "state": h[:, -1].clone()}
    if s["case"]["train"]:
        out["chunk_states"] = _kept(h, s["state"])
    return out


def _scan_backward(s):
    dt, form = s["x"].dtype, s["case"]["form"]
    h, a, rest = _hidden(s)
    first = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    d_h = s["d_y"].float()
    out = {}
    if s["gate"] is not None:
        g = s["gate"].float()
        sig = torch.sigmoid(g)
        out["gate"] = (d_h * h * (sig * (1 + g * (1 - sig)))).to(dt)
        d_h = d_h * (g * sig)
    if s["d_state"] is not None:
        d_h = d_h.clone()
        d_h[:, -1] += s["d_state"]
    # G_t = d_h_t + a_(t+1) G_(t+1): the same recurrence in reversed time
    later = torch.cat([torch.zeros_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    G = _recur(later, d_h.flip(1)).flip(1)
    if form == "logit":
        out["x"] = (G * rest).to(dt)
        out["f"] = (G * (before - s["x"].float()) * a * rest).to(dt)
    else:
        out["x"] = G.to(dt)
        out["f"] = (G * before * a).to(dt)
    out["state"] = a[:, 0] * G[:, 0]
    return out


def _scan_step(s):
    a, rest = _gates(s["f"], s["case"]["form"])
    x = s["x"].float()
    h = a * s["state"] + (rest * x if s["case"]["form"] == "logit" else x)
    y = h if s["gate"] is None else h * _swish(s["gate"])
    return {"y": y.to(s["x"].dtype), "state": h}


def _normed(v, kind):
    """v normalised over its last axis, and 1 / its spread."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    inv = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * inv, inv


def _normed_grad(d_hat, hat, inv, kind):
    back = d_hat - hat * (d_hat * hat).mean(-1, keepdim=True)
    if kind == "layer":
        back = back - d_hat.mean(-1, keepdim=True)
    return back * inv


def _norm_gate(s):
    z, _ = _normed(s["y"].float(), s["case"]["norm"])
    if s["case"]["token_major"]:
        z = z.transpose(1, 2)
    if s["gate"] is not None:
        z = z * _swish(s["gate"])
    return {"o": z.to(s["y"].dtype).contiguous()}


def _norm_gate_backward(s):
    kind, dt = s["case"]["norm"], s["y"].dtype
    z, inv = _normed(s["y"].float(), kind)
    d = s["d_o"].float()
    out = {}
    if s["gate"] is not None:
        g = s["gate"].float()
        sig = torch.sigmoid(g)
        zt = z.transpose(1, 2) if s["case"]["token_major"] else z
        out["gate"] = (d * zt * (sig * (1 + g * (1 - sig)))).to(dt)
        d = d * (g * sig)
    if s["case"]["token_major"]:
        d = d.transpose(1, 2)
    out["y"] = _normed_grad(d, z, inv, kind).to(dt).contiguous()
    return out


def _add_norm(s):
    c, dt = s["case"], s["x"].dtype
    u = s["x"].float()
    if c["post"] != "none":
        u, _ = _normed(u, c["post"])
    if s["w_post"] is not None:
        u = u * s["w_post"]
    r = c["alpha"] * s["residual"].float() + c["beta"] * u
    y = _normed(r, c["pre"])[0] * s["w_pre"]
    return {"residual": r.to(dt), "y": y.to(dt)}


def _add_norm_backward(s):
    c, dt = s["case"], s["x"].dtype
    hat, inv = _normed(s["residual"].float(), c["pre"])
    d_y = s["d_y"].float()
    out = {"w_pre": (d_y * hat).sum(0)}
    d_r = _normed_grad(d_y * s["w_pre"], hat, inv, c["pre"]) + s["d_res"].float()
    out["residual"] = (c["alpha"] * d_r).to(dt)
    d_u, x = c["beta"] * d_r, s["x"].float()
    hat = x
    if c["post"] != "none":
        hat, inv = _normed(x, c["post"])
    if s["w_post"] is not None:
        out["w_post"] = (d_u * hat).sum(0)
        d_u = d_u * s["w_post"]
    out["x"] = (_normed_grad(d_u, hat, inv, c["post"]) if c["post"] != "none" else d_u).to(dt)
    return out


# ---- the package's calls -----------------------------------------------------------

def _own(s):
    import linear_recurrent_sequence_scale_b200 as ret
    c, op = s["case"], s["case"]["op"]
    if op == "scan":
        got = ret.scan(s["x"], s["f"], form=c["form"], gate=s["gate"], state_in=s["state"],
                       return_state=True, return_chunk_states=c["train"])
        return dict(zip(("y", "state", "chunk_states"), got))
    if op == "scan_backward":
        gx, gf, gg, gs = ret.scan_backward(s["x"], s["f"], s["chunk_states"], s["d_y"],
                                           form=c["form"], gate=s["gate"],
                                           d_state_out=s["d_state"])
        return {"x": gx, "f": gf, "state": gs} | ({} if gg is None else {"gate": gg})
    if op == "scan_step":
        y = ret.scan_step(s["x"], s["f"], s["state"], form=c["form"], gate=s["gate"],
                          state_out=s["new_state"])
        return {"y": y, "state": s["new_state"]}
    if op == "norm_gate":
        return {"o": ret.norm_gate(s["y"], s["gate"], norm=c["norm"], eps=EPS,
                                   token_major=c["token_major"])}
    if op == "norm_gate_backward":
        gy, gg = ret.norm_gate_backward(s["y"], s["gate"], s["d_o"], norm=c["norm"], eps=EPS,
                                        token_major=c["token_major"])
        return {"y": gy} | ({} if gg is None else {"gate": gg})
    post = None if c["post"] == "none" else c["post"]
    if op == "add_norm":
        r, y = ret.add_norm(s["x"], s["residual"], s["w_pre"], w_post=s["w_post"],
                            post_norm=post, norm=c["pre"], alpha=c["alpha"], beta=c["beta"],
                            eps=EPS)
        return {"residual": r, "y": y}
    gx, gr, gpre, gpost = ret.add_norm_backward(
        s["x"], s["residual"], s["w_pre"], s["d_y"], s["d_res"], w_post=s["w_post"],
        post_norm=post, norm=c["pre"], alpha=c["alpha"], beta=c["beta"], eps=EPS)
    return {"x": gx, "residual": gr, "w_pre": gpre} | ({} if gpost is None else {"w_post": gpost})


_PLAIN = dict(scan=_scan, scan_backward=_scan_backward, scan_step=_scan_step,
              norm_gate=_norm_gate, norm_gate_backward=_norm_gate_backward, add_norm=_add_norm,
              add_norm_backward=_add_norm_backward)


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    g = int(bool(c.get("gate")))
    if c["op"] == "scan":
        n, chan = c["B"] * c["N"] * c["D"], c["B"] * c["D"]
        kept = chan * -(-c["N"] // CHUNK) if c["train"] else 0
        return {"bytes": n * es * (3 + g) + 4 * (chan * (1 + int(c["state"])) + kept),
                "flops": n * (8 + 5 * g)}
    if c["op"] == "scan_backward":
        n, chan = c["B"] * c["N"] * c["D"], c["B"] * c["D"]
        return {"bytes": n * es * (5 + 2 * g)
                + 4 * chan * (1 + int(c["state"]) + -(-c["N"] // CHUNK)),
                "flops": n * (16 + 12 * g)}
    if c["op"] == "scan_step":
        n = c["B"] * c["D"]
        return {"bytes": n * (es * (3 + g) + 8), "flops": n * (8 + 5 * g)}
    if c["op"] == "norm_gate":
        n = c["B"] * c["H"] * c["N"] * c["dv"]
        return {"bytes": n * es * (2 + g), "flops": n * (6 + 5 * g)}
    if c["op"] == "norm_gate_backward":
        n = c["B"] * c["H"] * c["N"] * c["dv"]
        return {"bytes": n * es * (3 + 2 * g), "flops": n * (14 + 12 * g)}
    n, d, w = c["rows"] * c["d"], c["d"], int(c["wpost"])
    two = int(c["post"] != "none")
    if c["op"] == "add_norm":
        return {"bytes": n * es * 4 + 4 * d * (1 + w), "flops": n * (9 + 5 * two + w)}
    reads = 3 + int(two or w)  # x only where its norm or its weight's gradient asks for it
    return {"bytes": n * es * (reads + 2) + 8 * d * (1 + w), "flops": n * (14 + 10 * two + 3 * w)}


# ---- the definitions in float64 -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    wide = lambda k: None if s.get(k) is None else s[k].double()  # noqa: E731
    if c["op"].startswith("scan"):
        return _exact_scan(c, {k: wide(k) for k in ("x", "f", "gate", "state", "d_y", "d_state")})
    leaf = lambda k: None if s.get(k) is None else s[k].double().requires_grad_()  # noqa: E731
    if c["op"].startswith("norm_gate"):
        y, g = leaf("y"), leaf("gate")
        with torch.set_grad_enabled(c["op"] == "norm_gate_backward"):
            o = _exact_norm(y, c["norm"])
            o = o.permute(0, 2, 1, 3) if c["token_major"] else o
            o = o if g is None else o * g / (1 + torch.exp(-g))
            if c["op"] == "norm_gate":
                return {"o": o.contiguous()}
            o.backward(s["d_o"].double())
        return {"y": y.grad} | ({} if g is None else {"gate": g.grad})
    if c["op"] == "add_norm":
        x, wpre, wpost = wide("x"), wide("w_pre"), wide("w_post")
        r = c["alpha"] * wide("residual") + c["beta"] * _exact_post(c, x, wpost)
        return {"residual": r, "y": _exact_norm(r, c["pre"]) * wpre}
    # The backward call is given the stored sum r: the gradient of y(r) and of r(residual, x).
    r, wpre = leaf("residual"), leaf("w_pre")
    (_exact_norm(r, c["pre"]) * wpre).backward(s["d_y"].double())
    d_r = r.grad + s["d_res"].double()
    x, wpost = leaf("x"), leaf("w_post")
    _exact_post(c, x, wpost).backward(c["beta"] * d_r)
    out = {"x": x.grad, "residual": c["alpha"] * d_r, "w_pre": wpre.grad}
    return out | ({} if wpost is None else {"w_post": wpost.grad})


def _exact_norm(v, kind):
    mean = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
    return (v - mean) / ((v - mean).pow(2).mean(-1, keepdim=True) + EPS).sqrt()


def _exact_post(c, x, w):
    u = x * 1.0 if c["post"] == "none" else _exact_norm(x, c["post"])
    return u if w is None else u * w


def _exact_scan(c, s):
    """Token after token, and back again for the gradients."""
    x, f, g = s["x"], s["f"], s["gate"]
    if c["form"] == "logit":
        a, rest = 1 / (1 + torch.exp(-f)), 1 / (1 + torch.exp(f))
        u = rest * x
    else:
        a, u = torch.exp(f), x
    swish = None if g is None else g / (1 + torch.exp(-g))
    if c["op"] == "scan_step":
        h = a * s["state"] + u
        return {"y": h if g is None else h * swish, "state": h}
    N = c["N"]
    h = torch.empty_like(x)
    past = torch.zeros_like(x[:, 0]) if s["state"] is None else s["state"]
    start = past
    for t in range(N):
        past = torch.addcmul(u[:, t], a[:, t], past)
        h[:, t] = past
    if c["op"] == "scan":
        out = {"y": h if g is None else h * swish, "state": past}
        if c["train"]:
            out["chunk_states"] = torch.stack(
                [start if t == 0 else h[:, t - 1] for t in range(0, N, CHUNK)], 1)
        return out
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    d_h = s["d_y"] if g is None else s["d_y"] * swish
    flow = torch.zeros_like(start) if s["d_state"] is None else s["d_state"]
    G = torch.empty_like(h)
    for t in range(N - 1, -1, -1):
        G[:, t] = d_h[:, t] + flow
        flow = a[:, t] * G[:, t]
    d_a = G * (before - x if c["form"] == "logit" else before)
    out = {"x": G * rest if c["form"] == "logit" else G,
           "f": d_a * a * rest if c["form"] == "logit" else d_a * a, "state": flow}
    if g is not None:
        sig = 1 / (1 + torch.exp(-g))
        out["gate"] = s["d_y"] * h * (sig + g * sig * (1 - sig))
    return out
