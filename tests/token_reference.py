"""Plain 64-bit implementations of the token operators, dense and loop-free,
on the CPU: what the kernels' tests compare with.  Each also returns the sums
of absolute terms that bound a kernel's rounding errors."""

import math

import numpy as np
import torch

LOW = np.uint64(0xFFFFFFFF)


def philox(counter, key):
    """Philox4x32-10: four arrays (broadcast together) and two words -> four uint64 arrays of 32-bit words."""
    c = [np.array(x, dtype=np.uint64) for x in np.broadcast_arrays(*counter)]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & LOW,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def numbers(counter, seed):
    """The eight 16-bit numbers of each call, along a last axis."""
    w = philox(counter, (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], -1).astype(np.int64)


def factors(n, ratio):
    """0 for a dropped element, 1 / (1 - p) for a kept one, p the ratio in 16 bits."""
    t = math.floor(np.float32(ratio).astype(np.float64) * 65536 + 0.5)
    return torch.from_numpy(np.where(n >= t, 65536.0 / (65536 - t), 0.0))


def dropout(x, ratio, seed, call, residual=None):
    n = x.numel()
    at = np.arange((n + 7) // 8, dtype=np.uint64)
    f = factors(numbers((at & LOW, at >> np.uint64(32), 0, call), seed).reshape(-1)[:n], ratio).reshape(x.shape)
    y = torch.where(f > 0, x.double() * f, 0.0)
    return y if residual is None else y + residual.double()


def layer_norm(x, scale, bias, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    inv = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - mean) * inv
    y = xh * scale.double() + (0 if bias is None else bias.double())
    return y, mean[..., 0], inv[..., 0], xh


def layer_norm_backward(dy, x, scale, eps):
    _, _, inv, xh = layer_norm(x, scale, None, eps)
    dy = dy.double()
    g = dy * scale.double()
    dx = inv[..., None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    flat = (-1, x.shape[-1])
    return dx, (dy * xh).reshape(flat).sum(0), dy.reshape(flat).sum(0)


def first_distances(n, max_distance):
    """First distance of each of n buckets of a side, in whole numbers."""
    e = n // 2
    starts = list(range(e))
    d = e
    for j in range(n - e):
        while d ** (n - e) * e ** j < max_distance ** j * e ** (n - e):
            d += 1
        starts.append(d)
    return starts


def bucket(rel, num_buckets, max_distance, bidirectional):
    rel = np.asarray(rel)
    n = num_buckets // 2 if bidirectional else num_buckets
    d = np.abs(rel) if bidirectional else np.maximum(-rel, 0)
    b = np.searchsorted(np.array(first_distances(n, max_distance)), d, side="right") - 1
    return b + np.where(rel > 0, n, 0) if bidirectional else b


def attention(q, k, v, scale, causal, lengths, table, max_distance, bidirectional, first, ratio, seed, call,
              do=None, u=0.0, tiny=0.0):
    """Outputs {"o", "lse"} and, with dO, {"dq", "dk", "dv", "dtable"}, each as (value, bound): the bound holds a
    kernel's error that accumulates in fp32, rounds P, dS and O to a type of unit roundoff `u`, and rounds each
    output once (to `u`); a rounding below the type's smallest normal number is off by up to `tiny`.  `first` is an
    int or one per sequence."""
    B, H, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    e = 2.0 ** -24
    lengths = torch.full((B,), Lk) if lengths is None else lengths.long().clamp(0, Lk)
    first = torch.as_tensor(first).expand(B)
    j = torch.arange(Lk)
    rel = j - (torch.arange(Lq)[:, None] + first[:, None, None])          # (B, Lq, Lk)
    seen = (j < lengths[:, None, None]).expand(B, Lq, Lk)
    if causal:
        seen = seen & (rel <= 0)
    seen = seen[:, None]
    held = (j < lengths[:, None])[:, None, :, None]
    G = H // Hkv
    q64 = q.double()
    k64, v64 = (torch.where(held, t.double(), 0.0).repeat_interleave(G, 1) for t in (k, v))
    s = q64 @ k64.transpose(-1, -2) * scale
    sa = q64.abs() @ k64.abs().transpose(-1, -2) * abs(scale)
    idx = None
    if table is not None:
        idx = torch.from_numpy(bucket(rel.numpy(), table.shape[0], max_distance, bidirectional))
        bias = table.double()[idx].permute(0, 3, 1, 2)
        s, sa = s + bias, sa + bias.abs()
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True) if Lk else torch.full((B, H, Lq, 1), -math.inf)
    top = torch.where(top == -math.inf, 0.0, top)
    x = torch.exp(s - top)
    total = x.sum(-1, keepdim=True)
    p = x / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, torch.log(total) + top, -math.inf)[..., 0]
    # a score's absolute error: its sum of D terms, the scale, the bias, the base-2 form and the exponential's
    # argument; the row's largest covers the maximum and the sum
    es = torch.where(seen, (D + 12) * e * sa, 0.0)
    es = es + es.amax(-1, keepdim=True) if Lk else es
    ep = es + (4 * (lse.abs().clamp(max=1e4)[..., None] + 1) + Lk / 8 + 24) * e  # relative, of a probability
    m = torch.ones(())
    if ratio > 0:
        at = np.arange((Lk + 7) // 8, dtype=np.uint64)
        rows = np.arange(Lq, dtype=np.uint64)[:, None]
        bh = np.arange(B * H, dtype=np.uint64)[:, None, None]
        m = factors(numbers((at, rows, bh, call), seed).reshape(B * H, Lq, -1)[..., :Lk], ratio).reshape(p.shape)
    w = p * m
    o = w @ v64
    # P is rounded before it is divided by the row's sum, which is at least 1
    eo = (w * (u + 2 * ep) + 2 * tiny * m * seen) @ v64.abs() + 4 * e * o.abs() + tiny
    res = {"o": (o, u * o.abs() + (1 + u) * eo), "lse": (lse, torch.where(
        total > 0, es.amax(-1, keepdim=True) + (6 * (lse.abs()[..., None].clamp(max=1e4) + 1) + Lk / 8) * e,
        0.0)[..., 0] if Lk else torch.zeros_like(lse))}
    if do is None:
        return res
    g = do.double()
    dp = g @ v64.transpose(-1, -2) * m
    dpa = g.abs() @ v64.abs().transpose(-1, -2) * m
    delta = (p * dp).sum(-1, keepdim=True)
    # delta is made from the rounded O
    ed = (g.abs() * (u * o.abs() + (1 + u) * eo)).sum(-1, keepdim=True) + (D + 8) * e * (
        g.abs() * o.abs()).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    eds = p * ((D + 8) * e * dpa + ed + 4 * e * (dp.abs() + delta.abs())) + ds.abs() * 2 * ep
    dsa = eds * (1 + u) + ds.abs() * u + tiny * seen                                    # of the rounded dS
    def shared(t):
        return t.reshape(B, Hkv, G, Lk, D).sum(2)
    n = max(Lq, Lk) * G
    dq = ds @ k64 * scale
    dk = shared(ds.transpose(-1, -2) @ q64 * scale)
    dv = shared(w.transpose(-1, -2) @ g)
    acc = (n + 8) * e
    bq = (dsa + acc * ds.abs()) @ k64.abs() * abs(scale)
    bk = shared((dsa + acc * ds.abs()).transpose(-1, -2) @ q64.abs() * abs(scale))
    bv = shared((w * (u + 2 * ep + acc) + tiny * m * seen).transpose(-1, -2) @ g.abs())
    for name, val, bnd in (("dq", dq, bq), ("dk", dk, bk), ("dv", dv, bv)):
        res[name] = (val, u * val.abs() + (1 + u) * bnd + tiny)
    if table is not None:
        nb = table.shape[0]
        dt, bt = torch.zeros(nb, H, dtype=torch.float64), torch.zeros(nb, H, dtype=torch.float64)
        for b in range(B):
            flat = idx[b].reshape(-1)
            dt.index_add_(0, flat, ds[b].reshape(H, -1).t())
            # a bucket's sum is made of short sums of at most 16 * Lk / 32 + 256 terms, then in double
            bt.index_add_(0, flat, (eds[b] + (Lk + 300) * e * ds[b].abs()).reshape(H, -1).t())
        ut = torch.finfo(table.dtype).eps / 2
        res["dtable"] = (dt, ut * dt.abs() + (1 + ut) * bt + (tiny if table.dtype != torch.float32 else 0.0))
    return res
