"""Plain 64-bit implementations of the gated projections, the norms around a
block and the gated recurrence, on the CPU.  With each value comes a bound on
the error of a kernel that works in fp32 and rounds where the header says, made
by carrying each rounding's error through the formulas: `e` is half a step of
fp32, `u` and `tiny` those of the output's type (relative, and below its
smallest normal number).  Products of two errors are left out: errors are below
2^-9 of their values in the tests, which SECOND covers."""

import math

import torch

E = 2.0 ** -24
SECOND = 1 + 2.0 ** -7


def unit(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return 2.0 ** -25 if t == torch.float16 else 2.0 ** -126


def rounded(value, err, t):
    """A value's bound once it is rounded to t."""
    return value, unit(t) * value.abs() + (1 + unit(t)) * SECOND * err + tiny(t)


# ------------------------------------------------------- gated projections

def activation(kind, a):
    """Value, slope, and the largest slope and curvature anywhere."""
    if kind == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s)), 1.1, 0.5
    if kind == "gelu":
        phi = 0.5 * torch.erfc(-a / math.sqrt(2))
        return a * phi, phi + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi), 1.13, 0.8
    if kind == "gelu_tanh":
        r = math.sqrt(2 / math.pi)
        th = torch.tanh(r * (a + 0.044715 * a ** 3))
        return (0.5 * a * (1 + th), 0.5 * (1 + th) + 0.5 * a * (1 - th * th) * r * (1 + 0.134145 * a * a), 1.13, 0.9)
    return a.clamp_min(0), (a > 0).double(), 1.0, 0.0


def gated(x, wg, wu, kind, dy=None):
    t = x.dtype
    x, wg, wu = x.double(), wg.double(), wu.double()
    rows, width, hidden = x.shape[0], x.shape[1], wg.shape[0]
    xa = x.abs()
    a, b = x @ wg.t(), x @ wu.t()
    ea, eb = ((width + 16) * E * (xa @ w.abs().t()) for w in (wg, wu))
    f, slope, steep, curved = activation(kind, a)
    # the exponential's argument is off by some roundings of itself: of a, of a^2 / 2 and of z, at most a^2 + 2 |a|
    own = 16 * E * (1 + a * a + a.abs()) * (f.abs() + 1e-30)
    ef = steep * ea + own
    y = f * b
    res = {"a": (a, SECOND * ea), "b": (b, SECOND * eb),
           "y": rounded(y, b.abs() * ef + f.abs() * eb + 4 * E * y.abs(), t)}
    if dy is None:
        return res
    dy = dy.double()
    es = torch.where(a.abs() <= 2 * ea, 1.0, 0.0) if kind == "relu" else (
        curved * ea + 24 * E * (1 + a * a + a.abs()) * (slope.abs() + f.abs() + torch.exp(-a * a / 2)))
    da, db = dy * b * slope, dy * f
    u = unit(t)
    eda = u * da.abs() + (1 + u) * SECOND * (dy.abs() * (b.abs() * es + eb * slope.abs()) + 6 * E * da.abs()) + tiny(t)
    edb = u * db.abs() + (1 + u) * SECOND * (dy.abs() * ef + 6 * E * db.abs()) + tiny(t)
    acc = (2 * hidden + 72) * E
    res["dx"] = rounded(da @ wg + db @ wu, (eda + acc * da.abs()) @ wg.abs() + (edb + acc * db.abs()) @ wu.abs(), t)
    acc = (rows + 72) * E
    for name, d, ed in (("dgate", da, eda), ("dup", db, edb)):
        res[name] = rounded(d.t() @ x, (ed + acc * d.abs()).t() @ xa, t)
    return res


# --------------------------------------------------- norms around a block

def norm(z, ez, layer, eps):
    """Normalised rows, the mean and the factor, each with its error (ez: that of z)."""
    n = z.shape[-1]
    chain = (n / 64 + 48) * E                         # relative error of a sum of n terms of one sign
    def mean(v):
        return v.mean(-1, keepdim=True)
    mu = mean(z) if layer else torch.zeros_like(z[..., :1])
    emu = mean(ez) + chain * mean(z.abs()) if layer else torch.zeros_like(mu)
    zc = z - mu
    ezc = ez + emu + E * zc.abs()
    var = mean(zc * zc) + eps
    inv = var.rsqrt()
    einv = inv * ((mean(zc.abs() * ezc) + chain * mean(zc * zc)) / var + 4 * E)
    # the mean's own error adds its square to the variance
    einv = einv + inv * emu * emu / (2 * var)
    zh = zc * inv
    return (zh, ezc * inv + zc.abs() * einv + 2 * E * zh.abs()), (mu, emu), (inv, einv)


def norm_gradient(g, eg, zh, ezh, inv, einv, layer):
    n = g.shape[-1]
    chain = (n / 64 + 48) * E
    def mean(v):
        return v.mean(-1, keepdim=True)
    c, ec = mean(g * zh), chain * mean((g * zh).abs()) + mean(eg * zh.abs() + g.abs() * ezh)
    a = mean(g) if layer else torch.zeros_like(c)
    ea = chain * mean(g.abs()) + mean(eg) if layer else torch.zeros_like(c)
    inner = g - a - zh * c
    einner = eg + ea + ezh * c.abs() + zh.abs() * ec + 4 * E * (g.abs() + a.abs() + (zh * c).abs())
    return inv * inner, inv * einner + einv * inner.abs() + 2 * E * (inv * inner).abs()


def join(x, branch, post, post_bias, pre, pre_bias, gate, alpha, eps, kind, dh=None, dy=None):
    """Everything residual_norm and its backward give, for x of (batch, tokens, cols)."""
    t, layer = x.dtype, kind == "layer"
    alpha = float(torch.tensor(alpha, dtype=torch.float32))
    eps = float(torch.tensor(eps, dtype=torch.float32))
    pt = next((v.dtype for v in (post, pre) if v is not None), t)
    x64, f = x.double(), branch.double()
    zero = torch.zeros_like(f)
    p, ep = f, zero
    m = torch.ones_like(f) if gate is None else gate.double()
    if gate is not None and 1 < gate.dim() < x.dim():
        m = m.reshape(*gate.shape[:-1], *([1] * (x.dim() - gate.dim())), x.shape[-1])
    m = m.expand(x.shape)
    stats = [torch.zeros(x.shape[:-1]).double(), torch.ones(x.shape[:-1]).double()] * 2
    estats = [torch.zeros(x.shape[:-1]).double()] * 4
    if post is not None:
        (fh, efh), (mu, emu), (finv, efinv) = norm(f, zero, layer, eps)
        w, b = post.double(), 0 if post_bias is None else post_bias.double()
        p = fh * w + b
        ep = efh * w.abs() + 3 * E * ((fh * w).abs() + (0 if post_bias is None else b.abs()))
        stats[:2], estats[:2] = [mu[..., 0], finv[..., 0]], [emu[..., 0] + E * mu[..., 0].abs(), efinv[..., 0]]
    h = alpha * x64 + m * p
    eh = m.abs() * ep + 3 * E * ((alpha * x64).abs() + (m * p).abs())
    res = {"h": rounded(h, eh, t)}
    if pre is not None:
        (hh, ehh), (mu, emu), (hinv, ehinv) = norm(h, eh, layer, eps)
        w, b = pre.double(), 0 if pre_bias is None else pre_bias.double()
        res["y"] = rounded(hh * w + b, ehh * w.abs() + 3 * E * ((hh * w).abs() + (
            0 if pre_bias is None else b.abs())), t)
        stats[2:], estats[2:] = [mu[..., 0], hinv[..., 0]], [emu[..., 0] + E * mu[..., 0].abs(), ehinv[..., 0]]
    res["stats"] = (torch.stack(stats, -1), SECOND * torch.stack(estats, -1))
    if dh is None and dy is None:
        return res
    def total(v, ev, like):
        """Sums over the axes that `like` lacks."""
        axes = tuple(range(like.dim() - 1, x.dim() - 1))
        if not axes:
            return rounded(v, ev, like.dtype)
        terms = math.prod(x.shape[i] for i in axes)
        return rounded(v.sum(axes), ev.sum(axes) + (terms + 32) * E * v.abs().sum(axes), like.dtype)
    d, ed = (zero, zero) if dh is None else (dh.double(), zero)
    if pre is not None:
        g = dy.double() * pre.double()
        dn, edn = norm_gradient(g, E * g.abs(), hh, ehh, hinv, ehinv, layer)
        like = torch.empty(x.shape[-1], dtype=pt)
        res["dpre"] = total(dy.double() * hh, dy.double().abs() * ehh + E * (dy.double() * hh).abs(), like)
        res["dpre_bias"] = total(dy.double(), zero, like)
        d, ed = d + dn, ed + edn + E * (d.abs() + dn.abs())
    res["dx"] = rounded(alpha * d, abs(alpha) * (ed + E * d.abs()), t)
    if gate is not None:
        res["dgate"] = total(d * p, ed * p.abs() + d.abs() * ep + 2 * E * (d * p).abs(), gate)
    k, ek = d * m, ed * m.abs() + E * (d * m).abs()
    if post is not None:
        like = torch.empty(x.shape[-1], dtype=pt)
        res["dpost"] = total(k * fh, ek * fh.abs() + k.abs() * efh + E * (k * fh).abs(), like)
        res["dpost_bias"] = total(k, ek, like)
        w = post.double()
        k, ek = norm_gradient(k * w, ek * w.abs() + E * (k * w).abs(), fh, efh, finv, efinv, layer)
    res["dbranch"] = rounded(k, ek, t)
    return res


# ------------------------------------------------------- gated recurrence

def recurrence(x, g, state=None, lengths=None, dy=None, dlast=None):
    """Values and bounds of everything gated_recurrence and its backward give."""
    t = x.dtype
    B, L, C = x.shape
    x64, g64 = x.double(), g.double()
    n = torch.full((B,), L) if lengths is None else lengths.long().clamp(0, L)
    held = (torch.arange(L) < n[:, None])[..., None].expand(B, L, C)
    x64, g64 = torch.where(held, x64, 0.0), torch.where(held, g64, 0.0)
    a, rest = torch.sigmoid(g64), torch.sigmoid(-g64)
    # the exponential's argument is rounded; a reciprocal and its products
    off = (1.5 * g64.abs() + 8) * E
    h = torch.zeros(B, C).double() if state is None else state.double()
    eh, ha = torch.zeros_like(h), h.abs()
    y, ey, before, ebefore = (torch.zeros(B, L, C).double() for _ in range(4))
    for i in range(L):
        k = held[:, i]
        before[:, i], ebefore[:, i] = h, eh + 64 * E * ha
        b = rest[:, i] * x64[:, i]
        eh = torch.where(k, a[:, i] * eh + (off[:, i] + 4 * E) * (a[:, i] * ha + b.abs()), eh)
        ha = torch.where(k, a[:, i] * ha + b.abs(), ha)
        h = torch.where(k, a[:, i] * h + b, h)
        y[:, i], ey[:, i] = torch.where(k, h, 0.0), torch.where(k, eh + 64 * E * ha, 0.0)
    res = {"y": rounded(y, ey, t), "last": (h, SECOND * (eh + 64 * E * ha) + tiny(torch.float32))}
    if dy is None:
        return res
    u = torch.zeros(B, C).double() if dlast is None else dlast.double()
    eu, ua = torch.zeros_like(u), u.abs()
    dx, edx, dg, edg = (torch.zeros(B, L, C).double() for _ in range(4))
    dy64 = torch.where(held, dy.double(), 0.0)
    for i in reversed(range(L)):
        k = held[:, i]
        D, eD, Da = dy64[:, i] + u, eu + 2 * E * (dy64[:, i].abs() + ua), dy64[:, i].abs() + ua
        eD = eD + 64 * E * Da
        ar, aa = rest[:, i], a[:, i]
        dx[:, i] = torch.where(k, ar * D, 0.0)
        edx[:, i] = torch.where(k, ar * (eD + (off[:, i] + 2 * E) * D.abs()), 0.0)
        gap = before[:, i] - x64[:, i]
        egap = ebefore[:, i] + E * (before[:, i].abs() + x64[:, i].abs())
        dg[:, i] = torch.where(k, D * gap * aa * ar, 0.0)
        edg[:, i] = torch.where(k, aa * ar * (eD * gap.abs() + D.abs() * egap + D.abs() * gap.abs() * (
            2 * off[:, i] + 6 * E)), 0.0)
        eu = torch.where(k, aa * (eu + (off[:, i] + 6 * E) * Da), eu)
        ua = torch.where(k, aa * Da, ua)
        u = torch.where(k, aa * D, u)
    res["dx"], res["dg"] = rounded(dx, edx, t), rounded(dg, edg, t)
    res["dstate"] = (u, SECOND * (eu + 64 * E * ua) + tiny(torch.float32))
    return res
