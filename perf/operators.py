"""Cases, plain forms and exact values of the token operators.

Layer normalisation with its gradients, dropout whose mask comes from a
counter, and attention with a learned relative position bias by buckets,
forward, backward and for single tokens.  Where `own` is true, run() makes the
package's calls; otherwise it computes the same in elementary torch operations.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------- cases

def _norm(name, rows, cols, dtype, params, train):
    c = {"op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "params": params, "train": train}
    return dict(c, name=name) if name else c


def _drop(name, count, dtype, ratio, residual):
    c = {"op": "dropout", "count": count, "dtype": dtype, "ratio": ratio, "residual": residual}
    return dict(c, name=name) if name else c


def _attn(name, batch, heads, kv_heads, q_len, kv_len, dim, dtype, causal, buckets, distance, ratio, train,
          ragged=False, empty=False, by_position=False):
    """`ragged`: each sequence has a length of its own; `empty`: the last one has length 0;
    `by_position`: Q, K, V lie in memory as (batch, position, head, dim)."""
    c = {"op": "attention", "batch": batch, "heads": heads, "kv_heads": kv_heads, "q_len": q_len,
         "kv_len": kv_len, "dim": dim, "dtype": dtype, "causal": causal, "buckets": buckets,
         "distance": distance, "ratio": ratio, "train": train, "ragged": ragged, "empty": empty,
         "by_position": by_position}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token's hidden state, normalised before a projection while generating
        _norm("norm one token bf16", 1, 1024, "bf16", "bf16", False),
        # a batch of feature vectors whose width no vector load divides, trained in fp32
        _norm("norm train odd f32", 4099, 777, "f32", "f32", True),
        # a training step's activations, half data with fp32 parameters
        _norm("norm train wide bf16", 16384, 2048, "bf16", "f32", True),
        # a small head's activations: a launch and little more
        _drop("dropout odd f32", 100003, "f32", 0.1, False),
        # a residual branch of a large batch: dropout, then the sum
        _drop("dropout residual bf16", 16384 * 2048, "bf16", 0.1, True),
        # one new token against a short cache of one sequence
        _attn("decode short f16", 1, 8, 8, 1, 77, 64, "f16", True, 32, 128, 0.0, False),
        # one new token for each of a batch of long caches of different lengths, shared heads
        _attn("decode ragged bf16", 16, 32, 8, 1, 8192, 128, "bf16", True, 32, 128, 0.0, False, ragged=True),
        # encoding ragged sequences of tokens of a feature map, both directions
        _attn("encode ragged bf16", 4, 16, 16, 1024, 1024, 64, "bf16", False, 32, 128, 0.0, False, ragged=True,
              by_position=True),
        # a training step in fp32 at odd sizes, one sequence without a token
        _attn("train odd f32", 3, 6, 3, 333, 401, 48, "f32", False, 32, 128, 0.1, True, ragged=True, empty=True),
        # a training step of a decoder's self-attention
        _attn("train causal bf16", 2, 16, 16, 2048, 2048, 64, "bf16", True, 32, 128, 0.1, True, by_position=True),
        # long sequences, shared heads, wide heads, both directions, no dropout
        _attn("train long f16", 1, 16, 4, 4096, 4096, 128, "f16", False, 64, 256, 0.0, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "dropout", "decode", "attention", "attention", "attention"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind == "norm":
        cols = _log(rng, 1, 9000)
        if rng.random() < 0.5:
            cols = (cols + 7) // 8 * 8
        rows = _log(rng, 1, max(1, min(40000, 16384 * 2048 // cols)))
        return _norm(None, rows, cols, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.6)
    if kind == "dropout":
        return _drop(None, _log(rng, 1, 16384 * 2048), dtype, rng.choice([0.0, 0.05, 0.1, 0.25, 0.5, 0.9]),
                     rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 4, 5])
    dim = rng.choice([8, 16, 20, 32, 40, 48, 63, 64, 64, 80, 96, 128, 128])
    buckets = rng.choice([0, 4, 8, 32, 32, 64, 320])
    distance = rng.choice([40, 100, 128, 128, 800]) if buckets <= 32 else rng.choice([256, 800])
    if kind == "decode":
        batch = _log(rng, 1, 16)
        kv_len = _log(rng, 1, min(16384, 16 * 8 * 8192 // (batch * kv_heads)))
        return _attn(None, batch, heads, kv_heads, rng.choice([1, 1, 1, 2, 5]), kv_len, dim, dtype, True, buckets,
                     distance, 0.0, False, ragged=rng.random() < 0.6, by_position=rng.random() < 0.5)
    q_len = _log(rng, 1, 2048)
    kv_len = q_len if rng.random() < 0.6 else _log(rng, 1, 2048)
    batch = rng.randint(1, max(1, min(6, 16 * 2048 * 2048 // (heads * max(q_len, 64) * max(kv_len, 64)))))
    causal = rng.random() < 0.5 and kv_len >= q_len
    return _attn(None, batch, heads, kv_heads, q_len, kv_len, dim, dtype, causal, buckets, distance,
                 rng.choice([0.0, 0.0, 0.1, 0.3]), rng.random() < 0.7, ragged=not causal and rng.random() < 0.5,
                 empty=rng.random() < 0.2, by_position=rng.random() < 0.5)


def _lengths(c):
    """Keys that each sequence of the batch holds."""
    full, n = c["kv_len"], c["batch"]
    lens = [full - (b * full * 3) // (4 * n) if c["ragged"] else full for b in range(n)]
    if c["empty"] and n > 1:
        lens[-1] = 0
    return lens


def _decodes(c):
    """The queries are the last tokens of each sequence (a cache is read); else query 0's position is a number."""
    return not c["train"] and c["causal"] and c["ragged"]


def _first(c):
    """Position of query 0 among the keys."""
    return c["kv_len"] - c["q_len"] if c["causal"] else 0


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0, dtype=t):
        return (torch.randn(shape, generator=g, device="cuda") * scale + mean).to(dtype)

    s = {"case": case, "seed": seed * 0x9E3779B97F4A7C15 % 2 ** 63}
    if case["op"] == "norm":
        p = TYPES[case["params"]]
        n = (case["rows"], case["cols"])
        s.update(x=normal(*n, scale=1.5, mean=0.3), scale=normal(n[1], scale=0.2, mean=1.0, dtype=p),
                 bias=normal(n[1], scale=0.2, dtype=p))
        if case["train"]:
            s["dy"] = normal(*n)
    elif case["op"] == "dropout":
        s["x"] = normal(case["count"])
        s["residual"] = normal(case["count"]) if case["residual"] else None
    else:
        def heads(n, length, scale=1.0):
            if case["by_position"]:
                return normal(case["batch"], length, n, case["dim"], scale=scale).transpose(1, 2)
            return normal(case["batch"], n, length, case["dim"], scale=scale)
        s.update(q=heads(case["heads"], case["q_len"]), k=heads(case["kv_heads"], case["kv_len"]),
                 v=heads(case["kv_heads"], case["kv_len"]), table=None, lengths=None, do=None)
        if case["buckets"]:
            s["table"] = normal(case["buckets"], case["heads"], scale=0.5)
        if case["ragged"] or case["empty"]:
            s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        if case["train"]:
            s["do"] = heads(case["heads"], case["q_len"])
    return s


# ------------------------------------------------------------- plain forms

def _philox(c0, c1, c2, call, seed):
    """Philox4x32-10 (Salmon et al., 2011) of the counter (c0, c1, c2, call) under a 64-bit key: eight 16-bit
    numbers in a last axis, low halves first."""
    low = 0xFFFFFFFF
    c0, c1, c2 = torch.broadcast_tensors(c0, c1, c2)
    c3 = torch.full_like(c0, call)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the 64-bit products; the sign is masked away
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return torch.stack([v for w in (c0, c1, c2, c3) for v in (w & 0xFFFF, w >> 16)], -1)


def _kept(numbers, ratio):
    """1 / (1 - p) where an element is kept, 0 where it is dropped, with p the ratio rounded to 16 bits."""
    t = int(math.floor(ratio * 65536 + 0.5))
    return torch.where(numbers >= t, 65536.0 / (65536 - t), 0.0)


def _bucket(rel, buckets, distance, both):
    """Bucket of key position minus query position: one for each of the nearest half of the distances, then
    borders that grow geometrically up to `distance`; a distance on a border opens the bucket."""
    n = buckets // 2 if both else buckets
    side = torch.where(rel > 0, n, 0) if both else torch.zeros_like(rel)
    d = rel.abs() if both else (-rel).clamp_min(0)
    near = n // 2
    far = torch.floor(torch.log(d.clamp_min(near).double() / near) / math.log(distance / near) * (n - near) + 1e-9)
    return side + torch.where(d < near, d, (near + far.long()).clamp_max(n - 1))


def _plain_norm(s):
    c = s["case"]
    x, w, b = s["x"].float(), s["scale"].float(), s["bias"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    inv = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + 1e-5)
    xh = xc * inv
    y = (xh * w + b).to(s["x"].dtype)
    if not c["train"]:
        return y
    dy = s["dy"].float()
    dxh = dy * w
    dx = inv * (dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True))
    return {"y": y, "mean": mean[:, 0], "inv_std": inv[:, 0], "dx": dx.to(y.dtype),
            "dscale": (dy * xh).sum(0).to(s["scale"].dtype), "dbias": dy.sum(0).to(s["scale"].dtype)}


def _plain_dropout(s):
    c, x = s["case"], s["x"]
    n = x.numel()
    blocks = torch.arange((n + 7) // 8, device=x.device)
    kept = _kept(_philox(blocks & 0xFFFFFFFF, blocks >> 32, torch.zeros_like(blocks), 3, s["seed"]), c["ratio"])
    y = torch.where(kept.flatten()[:n] > 0, x.float() * kept.flatten()[:n], 0.0)
    return (y if s["residual"] is None else y + s["residual"].float()).to(x.dtype)


def _plain_attention(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    b, h, m, n, d, g = c["batch"], c["heads"], c["q_len"], c["kv_len"], c["dim"], c["kv_heads"]
    scale = 1.0 / math.sqrt(d)
    pos = torch.arange(n, device=q.device)
    lens = s["lengths"].long() if s["lengths"] is not None else torch.full((b,), n, device=q.device)
    first = (lens - m if _decodes(c) else torch.full_like(lens, _first(c))).view(b, 1, 1, 1, 1)
    rel = pos - (torch.arange(m, device=q.device)[:, None] + first)  # (b, 1, 1, m, n)
    seen = (pos < lens.view(b, 1, 1, 1, 1)) & ((rel <= 0) if c["causal"] else True)
    held = (pos < lens[:, None]).view(b, 1, 1, n, 1)
    qf = q.float().reshape(b, g, h // g, m, d)
    kf, vf = (torch.where(held, t.float().unsqueeze(2), 0.0) for t in (k, v))  # (b, g, 1, n, d)
    score = torch.matmul(qf * scale, kf.transpose(-1, -2))
    if c["buckets"]:
        near = rel if _decodes(c) else rel[:1]
        bias = s["table"].float()[_bucket(near, c["buckets"], c["distance"], not c["causal"])]
        score += bias.squeeze(1).squeeze(1).permute(0, 3, 1, 2).reshape(-1, g, h // g, m, n)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    kept = 1.0
    if c["ratio"] > 0:
        at = torch.arange((n + 7) // 8, device=q.device)
        rows = torch.arange(m, device=q.device)[:, None]
        pairs = torch.arange(b * h, device=q.device)[:, None, None]
        kept = _kept(_philox(at, rows, pairs, 5, s["seed"]), c["ratio"]).flatten(-2)[..., :n].reshape(p.shape)
    pd = p * kept
    o = torch.matmul(pd, vf)
    out = o.reshape(b, h, m, d).to(q.dtype)
    if not c["train"]:
        return out
    do = s["do"].float().reshape(b, g, h // g, m, d)
    dp = torch.matmul(do, vf.transpose(-1, -2)) * kept
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    res = {"o": out, "dq": (torch.matmul(ds, kf) * scale).reshape(b, h, m, d).to(q.dtype),
           "dk": (torch.matmul(ds.transpose(-1, -2), qf) * scale).sum(2).to(q.dtype),
           "dv": torch.matmul(pd.transpose(-1, -2), do).sum(2).to(q.dtype)}
    if c["buckets"]:
        # rows padded and read one element shorter put equal distances under each other
        skew = torch.nn.functional.pad(ds.sum(0).reshape(h, m, n).flip(1), (0, m)).reshape(h, -1)
        sums = skew[:, :m * (m + n - 1)].reshape(h, m, m + n - 1).sum(1, dtype=torch.float64)
        index = _bucket(torch.arange(m + n - 1, device=q.device) - (m - 1) - _first(c), c["buckets"], c["distance"],
                        not c["causal"])
        dtable = torch.zeros(c["buckets"], h, dtype=torch.float64, device=q.device)
        res["dtable"] = dtable.index_add(0, index, sums.t()).to(s["table"].dtype)
    return res


def run(state):
    c = state["case"]
    if own:
        return _own(state)
    return {"norm": _plain_norm, "dropout": _plain_dropout, "attention": _plain_attention}[c["op"]](state)


# ------------------------------------------------------ the package's calls

def _own(s):
    import spatial_transformer_grid_amd as gs

    c = s["case"]
    if c["op"] == "norm":
        if not c["train"]:
            return gs.layer_norm(s["x"], s["scale"], s["bias"])
        y, mean, inv_std = gs.layer_norm(s["x"], s["scale"], s["bias"], return_stats=True)
        dx, dscale, dbias = gs.layer_norm_backward(s["dy"], s["x"], s["scale"], mean, inv_std)
        return {"y": y, "mean": mean, "inv_std": inv_std, "dx": dx, "dscale": dscale, "dbias": dbias}
    if c["op"] == "dropout":
        return gs.dropout(s["x"], c["ratio"], seed=s["seed"], call=3, residual=s["residual"])
    how = dict(causal=c["causal"], kv_lengths=s["lengths"], table=s["table"], max_distance=c["distance"],
               bidirectional=not c["causal"], q_position="end" if _decodes(c) else _first(c), ratio=c["ratio"],
               seed=s["seed"], call=5)
    if not c["train"]:
        return gs.attention(s["q"], s["k"], s["v"], **how)
    o, lse = gs.attention(s["q"], s["k"], s["v"], return_lse=True, **how)
    dq, dk, dv, dtable = gs.attention_backward(s["do"], s["q"], s["k"], s["v"], o, lse, **how)
    res = {"o": o, "dq": dq, "dk": dk, "dv": dv}
    return dict(res, dtable=dtable) if c["buckets"] else res


# -------------------------------------------------------------------- work

def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "norm":
        n, p = case["rows"] * case["cols"], case["cols"] * BYTES[case["params"]]
        if not case["train"]:
            return {"bytes": 2 * n * size + 2 * p, "flops": 8 * n}
        # x, dy -> y, dx; the parameters and their gradients; two numbers a row
        return {"bytes": 4 * n * size + 4 * p + 8 * case["rows"], "flops": 20 * n}
    if case["op"] == "dropout":
        return {"bytes": (3 if case["residual"] else 2) * case["count"] * size, "flops": 3 * case["count"]}
    m, n, d, h = case["q_len"], case["kv_len"], case["dim"], case["heads"]
    pairs = keys = 0
    for length in _lengths(case):
        first = length - m if _decodes(case) else _first(case)
        keys += length
        pairs += sum(max(0, min(length, first + i + 1)) for i in range(m)) if case["causal"] else m * length
    rows = case["batch"] * h * m * d * size
    table = case["buckets"] * h * size
    kv = keys * case["kv_heads"] * d * size
    if not case["train"]:
        return {"bytes": 2 * rows + 2 * kv + table, "flops": 4 * pairs * h * d}
    whole = case["batch"] * n * case["kv_heads"] * d * size
    return {"bytes": 4 * rows + 2 * kv + 2 * whole + 2 * table, "flops": 14 * pairs * h * d}


# ------------------------------------------------------- exact, in 64 bits

def _numbers(counter, seed):
    """The generator once more, on 16-bit limbs: counter is a list of four int64 tensors of one shape."""
    def product(word, constant):
        lo = (word & 0xFFFF) * constant
        mid = (word >> 16) * constant + (lo >> 16)
        return mid >> 16, (mid & 0xFFFF) << 16 | lo & 0xFFFF
    x, key = list(counter), [seed % 2 ** 32, seed // 2 ** 32]
    for r in range(10):
        (h0, l0), (h1, l1) = product(x[0], 0xD2511F53), product(x[2], 0xCD9E8D57)
        ks = [(key[0] + r * 0x9E3779B9) % 2 ** 32, (key[1] + r * 0xBB67AE85) % 2 ** 32]
        x = [h1 ^ x[1] ^ ks[0], l1, h0 ^ x[3] ^ ks[1], l0]
    out = torch.empty(*x[0].shape, 8, dtype=torch.int64, device=x[0].device)
    for i in range(8):
        out[..., i] = (x[i // 2] >> (16 * (i % 2))) % 65536
    return out.reshape(*x[0].shape[:-1], -1)


def _borders(n, distance):
    """Smallest distance of each bucket of one side, from whole numbers: bucket near + j begins where
    (d / near) ** (n - near) reaches (distance / near) ** j."""
    near = n // 2
    m, starts = n - near, list(range(near))
    for j in range(m):
        lo, hi = near, distance
        while lo < hi:
            mid = (lo + hi) // 2
            if mid ** m * near ** j >= distance ** j * near ** m:
                hi = mid
            else:
                lo = mid + 1
        starts.append(lo)
    return starts


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        inv = (var + 1e-5).rsqrt()
        xh = (x - mean[:, None]) * inv[:, None]
        y = torch.addcmul(s["bias"].double(), xh, s["scale"].double())
        if not case["train"]:
            return y
        dy = s["dy"].double()
        gh = dy * s["scale"].double()
        n = case["cols"]
        dx = (gh - (gh.sum(1) / n)[:, None] - xh * ((gh * xh).sum(1) / n)[:, None]) * inv[:, None]
        return {"y": y, "mean": mean, "inv_std": inv, "dx": dx, "dscale": torch.linalg.vecdot(dy, xh, dim=0),
                "dbias": dy.sum(0)}
    if case["op"] == "dropout":
        x = s["x"].double()
        block = torch.arange(-(-case["count"] // 8), device="cuda")
        zero = torch.zeros_like(block)
        r = _numbers([block, zero, zero, zero + 3], s["seed"])[:case["count"]]
        p = round(case["ratio"] * 65536) / 65536
        y = x / (1 - p) * (r >= p * 65536)
        return y if s["residual"] is None else y + s["residual"].double()
    c, lens = case, _lengths(case)
    m, n, h, g, both = c["q_len"], c["kv_len"], c["heads"], c["kv_heads"], not c["causal"]
    index = torch.zeros(0)
    q, k, v = (s[x].double() for x in "qkv")
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dtable = torch.zeros(h, max(1, c["buckets"]), dtype=torch.float64, device="cuda")
    if c["buckets"]:
        side = c["buckets"] // 2 if both else c["buckets"]
        starts = torch.tensor(_borders(side, c["distance"]), device="cuda")
    for b, length in enumerate(lens):
        first = length - m if _decodes(c) else _first(c)
        if length == 0:
            continue
        i = torch.arange(first, first + m, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None]
        hidden = (j > i) if c["causal"] else torch.zeros(m, length, dtype=torch.bool, device="cuda")
        if c["buckets"]:
            away = (j - i).abs() if both else (i - j).clamp(min=0)
            index = torch.searchsorted(starts, away, right=True) - 1 + (side * (j > i) if both else 0)
        for a in range(h):
            kk, vv = k[b, a * g // h, :length], v[b, a * g // h, :length]
            z = q[b, a] @ kk.T / math.sqrt(c["dim"])
            if c["buckets"]:
                z = z + s["table"][:, a].double()[index]
            z = z.masked_fill(hidden, -math.inf)
            p = torch.softmax(z, 1).nan_to_num(0.0)
            w = p
            if c["ratio"]:
                at = torch.arange(-(-length // 8), device="cuda")[None].expand(m, -1)
                row = torch.arange(m, device="cuda")[:, None].expand_as(at)
                fixed = torch.zeros_like(at)
                r = _numbers([at, row, fixed + (b * h + a), fixed + 5], s["seed"])[:, :length]
                cut = round(c["ratio"] * 65536)
                keep = (r >= cut) / (1 - cut / 65536)
                w = p * keep
            o[b, a] = w @ vv
            if c["train"]:
                do = s["do"][b, a].double()
                dw = do @ vv.T
                if c["ratio"]:
                    dw = dw * keep
                dz = p * (dw - (p * dw).sum(1, keepdim=True))
                dq[b, a] = dz @ kk / math.sqrt(c["dim"])
                dk[b, a * g // h, :length] += dz.T @ q[b, a] / math.sqrt(c["dim"])
                dv[b, a * g // h, :length] += w.T @ do
                if c["buckets"]:
                    dtable[a] += torch.bincount(index.flatten(), dz.flatten(), c["buckets"])
    if not c["train"]:
        return o
    res = {"o": o, "dq": dq, "dk": dk, "dv": dv}
    return dict(res, dtable=dtable.T.contiguous()) if c["buckets"] else res
