"""Cases, plain forms and exact values of the operators of a gated block.

The gated feed-forward projections, the norms before and after a block joined
with its gate and residual, and a gated linear recurrence along the tokens,
each with its gradients.  Where `own` is true, run() makes the package's calls;
otherwise it computes the same in elementary torch operations.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------- cases

def _gated(name, rows, width, hidden, dtype, activation, train):
    c = {"op": "gated", "rows": rows, "width": width, "hidden": hidden, "dtype": dtype, "activation": activation,
         "train": train}
    return dict(c, name=name) if name else c


def _join(name, batch, tokens, cols, dtype, params, norm, post, pre, gate, residual_scale, train):
    """`post`, `pre`: whether the branch and the sum are normalised; `gate`: none, or one row of it for all
    tokens (channel), for each sequence (sequence) or for each token (token)."""
    c = {"op": "join", "batch": batch, "tokens": tokens, "cols": cols, "dtype": dtype, "params": params, "norm": norm,
         "post": post, "pre": pre, "gate": gate, "residual_scale": residual_scale, "train": train}
    return dict(c, name=name) if name else c


def _scan(name, batch, length, channels, dtype, gate_mean, state, ragged, empty, train):
    """`state`: the sequences begin at a given state; `ragged`: each has a length of its own; `empty`: the last
    one has no token."""
    c = {"op": "scan", "batch": batch, "length": length, "channels": channels, "dtype": dtype,
         "gate_mean": gate_mean, "state": state, "ragged": ragged, "empty": empty, "train": train}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the feed-forward projections of one new token while generating
        _gated("gated one token bf16", 1, 1024, 4096, "bf16", "silu", False),
        # one new token for each of a batch of sequences
        _gated("gated decode f16", 16, 2048, 8192, "f16", "gelu_tanh", False),
        # a training step in fp32 at sizes that no vector load and no tile divides
        _gated("gated train odd f32", 577, 203, 531, "f32", "gelu", True),
        # the tokens of a few feature maps of odd extents, encoded
        _gated("gated encode f16", 4097, 1024, 2736, "f16", "gelu", False),
        # a training step of a large batch
        _gated("gated train bf16", 8192, 2048, 8192, "bf16", "silu", True),
        # one token's residual stream between two blocks while generating
        _join("join one token bf16", 1, 1, 1024, "bf16", "bf16", "rms", True, True, "none", 1.0, False),
        # a training step in fp32, a gate for each sequence, a width that no vector load divides
        _join("join train odd f32", 3, 1367, 777, "f32", "f32", "layer", True, True, "sequence", 1.25, True),
        # a training step's activations, half data with fp32 parameters and a gate for each channel
        _join("join train wide bf16", 8, 2048, 2048, "bf16", "f32", "rms", True, True, "channel", 1.0, True),
        # one new token for each of a batch of sequences, whose states are kept
        _scan("scan step f16", 16, 1, 2048, "f16", 2.0, True, False, False, False),
        # a training step in fp32, sequences of different lengths, one without a token
        _scan("scan train odd f32", 5, 1025, 190, "f32", 1.0, True, True, True, True),
        # one large feature map of 256 x 256 positions, read as a sequence of few channels
        _scan("scan one map f16", 1, 65536, 256, "f16", 3.0, False, False, False, False),
        # a training step of a batch of long sequences
        _scan("scan train long bf16", 4, 16384, 1024, "bf16", 3.0, False, False, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, n):
    return (n + 7) // 8 * 8 if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["gated", "gated", "join", "scan"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "gated":
        width, hidden = _eights(rng, _log(rng, 8, 2048)), _eights(rng, _log(rng, 8, 8192))
        most = 8192 * 2048 * 8192 // (8 if dtype == "f32" else 1)
        rows = _log(rng, 1, max(1, min(8192, most // (width * hidden))))
        return _gated(None, rows, width, hidden, dtype, rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                      rng.random() < 0.6)
    if op == "join":
        cols = _eights(rng, _log(rng, 16, 9000))
        batch = _log(rng, 1, 32)
        tokens = _log(rng, 1, max(1, min(4000, 8 * 2048 * 2048 // (batch * cols))))
        post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return _join(None, batch, tokens, cols, dtype, rng.choice([dtype, "f32"]), rng.choice(["rms", "layer"]), post,
                     pre, rng.choice(["none", "channel", "sequence", "token"]), rng.choice([1.0, 1.0, 0.5, 1.7]),
                     rng.random() < 0.6)
    batch = _log(rng, 1, 32)
    channels = _eights(rng, _log(rng, 1, 4096))
    length = _log(rng, 1, max(1, min(65536, 4 * 16384 * 1024 // (batch * channels))))
    return _scan(None, batch, length, channels, dtype, rng.choice([0.0, 1.0, 2.0, 3.0, 5.0]), rng.random() < 0.5,
                 rng.random() < 0.4, rng.random() < 0.2, rng.random() < 0.6)


def _lengths(c):
    """Tokens that each sequence of the batch holds."""
    full, n = c["length"], c["batch"]
    lens = [full - (b * full * 3) // (4 * n) if c["ragged"] else full for b in range(n)]
    if c["empty"] and n > 1:
        lens[-1] = 0
    return lens


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0, dtype=t):
        return (torch.randn(shape, generator=g, device="cuda") * scale + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "gated":
        m, k, n = case["rows"], case["width"], case["hidden"]
        s.update(x=normal(m, k), gate=normal(n, k, scale=k ** -0.5), up=normal(n, k, scale=k ** -0.5))
        if case["train"]:
            s["dy"] = normal(m, n)
    elif case["op"] == "join":
        p, n = TYPES[case["params"]], case["cols"]
        shape = (case["batch"], case["tokens"], n)
        s.update(x=normal(*shape, mean=0.2), branch=normal(*shape, scale=0.7, mean=0.1), gate=None)
        for name in ("post", "pre"):
            s[name] = normal(n, scale=0.2, mean=1.0, dtype=p) if case[name] else None
            s[name + "_bias"] = normal(n, scale=0.2, dtype=p) if case[name] and case["norm"] == "layer" else None
        lead = {"none": None, "channel": (), "sequence": shape[:1], "token": shape[:2]}[case["gate"]]
        if lead is not None:
            s["gate"] = normal(*lead, n, scale=0.5, mean=0.5, dtype=p)
        if case["train"]:
            s["dh"] = normal(*shape)
            s["dy"] = normal(*shape) if case["pre"] else None
    else:
        b, n, c = case["batch"], case["length"], case["channels"]
        s.update(x=normal(b, n, c), g=normal(b, n, c, scale=1.5, mean=case["gate_mean"]), state=None, lengths=None)
        if case["state"]:
            s["state"] = normal(b, c, dtype=torch.float32)
        if case["ragged"] or case["empty"]:
            s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        if case["train"]:
            s["dy"], s["dstate"] = normal(b, n, c), normal(b, c, dtype=torch.float32)
    return s


# ------------------------------------------------------------- plain forms

def _activation(name, a):
    """The activation of a and its slope."""
    if name == "silu":
        e = 1.0 / (1.0 + torch.exp(-a))
        return a * e, e * (1.0 + a * (1.0 - e))
    if name == "gelu":
        phi = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
        return a * phi, phi + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        r = math.sqrt(2.0 / math.pi)
        th = torch.tanh(r * (a + 0.044715 * a * a * a))
        return 0.5 * a * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * a * (1.0 - th * th) * r * (1.0 + 0.134145 * a * a)
    return a.clamp_min(0.0), (a > 0).float()


def _plain_gated(s):
    c, t = s["case"], s["x"].dtype
    x, wg, wu = s["x"].float(), s["gate"].float(), s["up"].float()
    a, b = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
    f, slope = _activation(c["activation"], a)
    y = (f * b).to(t)
    if not c["train"]:
        return y
    dy = s["dy"].float()
    da, db = dy * b * slope, dy * f
    return {"y": y, "dx": (torch.matmul(da, wg) + torch.matmul(db, wu)).to(t),
            "dgate": torch.matmul(da.t(), x).to(t), "dup": torch.matmul(db.t(), x).to(t)}


def _normalised(kind, x):
    """x normalised along its last axis, and the factor that its deviations have in it."""
    xc = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    inv = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + 1e-5)
    return xc * inv, inv


def _normalised_gradient(kind, d, xh, inv):
    """Gradient of x from that of its normalised values."""
    d = d - xh * (d * xh).mean(-1, keepdim=True)
    return inv * (d - d.mean(-1, keepdim=True) if kind == "layer" else d)


def _sum_to(t, like):
    """t summed over its tokens and, where `like` has no axis for them, its sequences."""
    t = t.double()
    t = t.sum(1) if like.dim() < 3 else t
    return (t.sum(0) if like.dim() < 2 else t).to(like.dtype)


def _plain_join(s):
    c, t, kind = s["case"], s["x"].dtype, s["case"]["norm"]
    f, gate = s["branch"].float(), s["gate"]
    m = 1.0
    if gate is not None:
        m = gate.float().unsqueeze(1) if gate.dim() == 2 else gate.float()
    if c["post"]:
        fh, finv = _normalised(kind, f)
        f = fh * s["post"].float() + (0.0 if s["post_bias"] is None else s["post_bias"].float())
    h = c["residual_scale"] * s["x"].float() + m * f
    res = {"h": h.to(t)}
    if c["pre"]:
        hh, hinv = _normalised(kind, h)
        res["y"] = (hh * s["pre"].float() + (0.0 if s["pre_bias"] is None else s["pre_bias"].float())).to(t)
    if not c["train"]:
        return res
    dh = s["dh"].float()
    if c["pre"]:
        dy = s["dy"].float()
        dh = dh + _normalised_gradient(kind, dy * s["pre"].float(), hh, hinv)
        res["dpre"] = _sum_to(dy * hh, s["pre"])
        if s["pre_bias"] is not None:
            res["dpre_bias"] = _sum_to(dy, s["pre"])
    res["dx"] = (c["residual_scale"] * dh).to(t)
    if gate is not None:
        res["dgate"] = _sum_to(dh * f, gate)
    df = dh * m
    if c["post"]:
        res["dpost"] = _sum_to(df * fh, s["post"])
        if s["post_bias"] is not None:
            res["dpost_bias"] = _sum_to(df, s["post"])
        df = _normalised_gradient(kind, df * s["post"].float(), fh, finv)
    res["dbranch"] = df.to(t)
    return res


def _running(a, b):
    """h_t = a_t h_(t-1) + b_t along axis 1 from zero: pairs of steps are one step of a sequence half as long."""
    n = a.shape[1]
    if n == 1:
        return b
    m = n // 2 * 2
    odd = _running(a[:, 1:m:2] * a[:, 0:m:2], a[:, 1:m:2] * b[:, 0:m:2] + b[:, 1:m:2])
    h = torch.empty_like(b)
    h[:, 1:m:2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :(n - 1) // 2] + b[:, 2::2]
    return h


def _plain_scan(s):
    c, t = s["case"], s["x"].dtype
    x, g = s["x"].float(), s["g"].float()
    n = c["length"]
    a, rest = 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))
    held = None
    if s["lengths"] is not None:  # past its length a sequence keeps its state
        held = (torch.arange(n, device=x.device) < s["lengths"][:, None]).unsqueeze(-1)
        a, rest, x = torch.where(held, a, 1.0), torch.where(held, rest, 0.0), torch.where(held, x, 0.0)
    first = torch.zeros_like(x[:, 0]) if s["state"] is None else s["state"]
    b = rest * x
    b[:, 0] += a[:, 0] * first
    h = _running(a, b)
    y = h if held is None else torch.where(held, h, 0.0)
    res = {"y": y.to(t), "state": h[:, -1].contiguous()}
    if not c["train"]:
        return res
    dy = s["dy"].float()
    d = dy.clone() if held is None else torch.where(held, dy, 0.0)
    d[:, -1] += s["dstate"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    d = _running(later.flip(1), d.flip(1)).flip(1)
    before = torch.cat([first.unsqueeze(1), h[:, :-1]], 1)
    res.update(dx=(d * rest).to(t), dg=(d * (before - x) * a * rest).to(t), dfirst=a[:, 0] * d[:, 0])
    return res


def run(state):
    c = state["case"]
    if own:
        return _own(state)
    return {"gated": _plain_gated, "join": _plain_join, "scan": _plain_scan}[c["op"]](state)


# ------------------------------------------------------ the package's calls

def _own(s):
    import spatial_transformer_grid_amd as gs

    c = s["case"]
    if c["op"] == "gated":
        if not c["train"]:
            return gs.gated_linear(s["x"], s["gate"], s["up"], c["activation"])
        y, saved = gs.gated_linear(s["x"], s["gate"], s["up"], c["activation"], return_saved=True)
        dx, dgate, dup = gs.gated_linear_backward(s["dy"], s["x"], s["gate"], s["up"], saved, c["activation"])
        return {"y": y, "dx": dx, "dgate": dgate, "dup": dup}
    if c["op"] == "join":
        how = dict(post_scale=s["post"], post_bias=s["post_bias"], pre_scale=s["pre"], gate=s["gate"],
                   residual_scale=c["residual_scale"], norm=c["norm"])
        if not c["train"]:
            h, y = gs.residual_norm(s["x"], s["branch"], pre_bias=s["pre_bias"], **how)
            return {"h": h, "y": y} if c["pre"] else {"h": h}
        h, y, stats = gs.residual_norm(s["x"], s["branch"], pre_bias=s["pre_bias"], return_stats=True, **how)
        dx, dbranch, dgate, dpost, dpost_bias, dpre, dpre_bias = gs.residual_norm_backward(
            s["dh"], s["dy"], s["x"], s["branch"], stats, **how)
        layer = c["norm"] == "layer"
        res = {"h": h, "dx": dx, "dbranch": dbranch}
        for name, value, there in (("y", y, c["pre"]), ("dgate", dgate, s["gate"] is not None),
                                   ("dpost", dpost, c["post"]), ("dpost_bias", dpost_bias, c["post"] and layer),
                                   ("dpre", dpre, c["pre"]), ("dpre_bias", dpre_bias, c["pre"] and layer)):
            if there:
                res[name] = value
        return res
    if not c["train"]:
        y, state = gs.gated_recurrence(s["x"], s["g"], s["state"], s["lengths"])
        return {"y": y, "state": state}
    y, state, saved = gs.gated_recurrence(s["x"], s["g"], s["state"], s["lengths"], return_saved=True)
    dx, dg, dfirst = gs.gated_recurrence_backward(s["dy"], s["x"], s["g"], saved, s["dstate"], s["lengths"])
    return {"y": y, "state": state, "dx": dx, "dg": dg, "dfirst": dfirst}


# -------------------------------------------------------------------- work

def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "gated":
        m, k, n = case["rows"], case["width"], case["hidden"]
        if not case["train"]:
            return {"bytes": (m * k + 2 * n * k + m * n) * size, "flops": 4 * m * n * k}
        # x, the weights, dy -> y, dx and the weights' gradients; six products
        return {"bytes": (2 * m * k + 4 * n * k + 2 * m * n) * size, "flops": 12 * m * n * k}
    if case["op"] == "join":
        n, p = case["batch"] * case["tokens"] * case["cols"], BYTES[case["params"]]
        rows = {"none": 0, "channel": 1, "sequence": case["batch"], "token": case["batch"] * case["tokens"]}
        rows = rows[case["gate"]] + (2 if case["norm"] == "layer" else 1) * (case["post"] + case["pre"])
        small = rows * case["cols"] * p
        if not case["train"]:
            return {"bytes": (3 + case["pre"]) * n * size + small, "flops": 14 * n}
        # x, branch, dh, dy -> h, y, dx, dbranch; the parameters and the gate, and their gradients
        return {"bytes": (6 + 2 * case["pre"]) * n * size + 2 * small, "flops": 40 * n}
    n = sum(_lengths(case)) * case["channels"]
    whole = case["batch"] * case["length"] * case["channels"]
    states = case["batch"] * case["channels"] * 4
    if not case["train"]:
        return {"bytes": (2 * n + whole) * size + (1 + case["state"]) * states, "flops": 8 * n}
    # x, gates, dy of the tokens there are -> y, dx, dg, zeros past a length; the states at both ends
    return {"bytes": (3 * n + 3 * whole) * size + (3 + case["state"]) * states, "flops": 24 * n}


# ------------------------------------------------------- exact, in 64 bits

def _exact_gated(s):
    c = s["case"]
    x, wg, wu = (s[n].double().requires_grad_(c["train"]) for n in ("x", "gate", "up"))
    a, fn = x @ wg.T, torch.nn.functional
    act = {"silu": fn.silu, "gelu": fn.gelu, "gelu_tanh": lambda v: fn.gelu(v, approximate="tanh"), "relu": fn.relu}
    y = act[c["activation"]](a) * (x @ wu.T)
    if not c["train"]:
        return y
    dx, dgate, dup = torch.autograd.grad(y, (x, wg, wu), s["dy"].double())
    return {"y": y.detach(), "dx": dx, "dgate": dgate, "dup": dup}


def _exact_join(s):
    c = s["case"]
    names = [n for n in ("x", "branch", "gate", "post", "post_bias", "pre", "pre_bias") if s[n] is not None]
    v = {n: s[n].double().requires_grad_(c["train"]) for n in names}

    def norm(z, which):
        w, b = v[which], v.get(which + "_bias")
        if c["norm"] == "layer":
            return torch.nn.functional.layer_norm(z, w.shape, w, b, 1e-5)
        return z / torch.sqrt((z ** 2).mean(-1, keepdim=True) + 1e-5) * w
    f = norm(v["branch"], "post") if c["post"] else v["branch"]
    if c["gate"] == "sequence":
        f = f * v["gate"][:, None]
    elif c["gate"] != "none":
        f = f * v["gate"]
    h = v["x"] * c["residual_scale"] + f
    out, back = [h], [s["dh"].double()] if c["train"] else []
    res = {"h": h.detach()}
    if c["pre"]:
        out.append(norm(h, "pre"))
        res["y"] = out[1].detach()
    if not c["train"]:
        return res
    back += [s["dy"].double()] if c["pre"] else []
    got = dict(zip(names, torch.autograd.grad(out, [v[n] for n in names], back)))
    order = ("pre", "pre_bias", "x", "gate", "post", "post_bias", "branch")
    return dict(res, **{"d" + n: got[n] for n in order if n in got})


def _steps(a, b, first):
    """States after each step along axis 0, a block of 256 steps at a time: all blocks step by step from zero, then
    from block to block, then what a block's first state adds."""
    n, size = a.shape[0], 256
    blocks = -(-n // size)
    if blocks * size > n:
        more = [blocks * size - n, *a.shape[1:]]
        a, b = torch.cat([a, a.new_ones(more)]), torch.cat([b, b.new_zeros(more)])
    a, b = (t.reshape(blocks, size, *t.shape[1:]) for t in (a, b))
    local, through = torch.empty_like(a), torch.empty_like(a)
    h, p = torch.zeros_like(a[:, 0]), torch.ones_like(a[:, 0])
    for i in range(size):
        h, p = a[:, i] * h + b[:, i], p * a[:, i]
        local[:, i], through[:, i] = h, p
    for j in range(blocks):
        local[j] += through[j] * first
        first = local[j, -1]
    return local.flatten(0, 1)[:n]


def _exact_scan(s):
    c = s["case"]
    y, dx, dg = (torch.zeros_like(s["x"], dtype=torch.float64) for _ in range(3))
    state = torch.zeros(c["batch"], c["channels"], dtype=torch.float64, device="cuda")
    state = state if s["state"] is None else s["state"].double()
    last, dfirst = state.clone(), torch.zeros_like(state)
    if c["train"]:
        dfirst = s["dstate"].double()
    for i, n in enumerate(_lengths(c)):
        if n == 0:
            continue
        x, g = s["x"][i, :n].double(), s["g"][i, :n].double()
        a = torch.sigmoid(g)
        h = _steps(a, torch.sigmoid(-g) * x, state[i])
        y[i, :n], last[i] = h, h[-1]
        if c["train"]:
            d = s["dy"][i, :n].double()
            d[-1] += s["dstate"][i]
            d = _steps(torch.cat([a[:1], a[1:].flip(0)]), d.flip(0), torch.zeros_like(state[i])).flip(0)
            dx[i, :n] = d * torch.sigmoid(-g)
            dg[i, :n] = d * (torch.cat([state[i:i + 1], h[:-1]]) - x) * a * torch.sigmoid(-g)
            dfirst[i] = d[0] * a[0]
    if not c["train"]:
        return {"y": y, "state": last}
    return {"y": y, "state": last, "dx": dx, "dg": dg, "dfirst": dfirst}


def exact(case, seed):
    return {"gated": _exact_gated, "join": _exact_join, "scan": _exact_scan}[case["op"]](prepare(case, seed))
