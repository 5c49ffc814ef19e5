"""The token operators on the GPU against the 64-bit reference, at the sizes,
layouts and masks where they can go wrong.  Every bound is derived from the
roundings a kernel makes (token_reference), none from a run."""

import math

import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def gs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import spatial_transformer_grid_amd as gs

    gs.token_lib()
    return gs


def unit(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return 2.0 ** -25 if t == torch.float16 else 0.0


def close(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, 0.0, (got - want).abs())
    bad = ~(off <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g times the bound" % (
        what, int(bad.sum()), bad.numel(), float((off / bound.clamp_min(1e-300))[bad].max()))


# ------------------------------------------------------------------ norm

def norm_bounds(x, w, b, dy, eps, t, pt):
    """Values and bounds of everything layer_norm and its backward give."""
    u, n, rows = unit(t), x.shape[-1], x.numel() // x.shape[-1]
    y, mean, inv, xh = ref.layer_norm(x, w, b, eps)
    xa, w64 = x.double().abs(), w.double()
    chain = (n / 64 + 32) * E32                      # relative error of a sum of n terms of one sign
    em = chain * xa.mean(-1)                         # of the mean
    # (x - mean): the mean's error and a rounding; inv_std: half the variance's relative error
    ev = chain + 2 * (em * inv) ** 2 + 8 * E32
    einv = ev + 4 * E32
    exh = (em[..., None] + E32 * (xa + mean.abs()[..., None])) * inv[..., None] + xh.abs() * (einv[..., None] + 2 * E32)
    res = {"y": (y, u * y.abs() + (1 + u) * (exh * w64.abs() + 4 * E32 * ((xh * w64).abs() + (
        0 if b is None else b.double().abs()))) + tiny(t)), "mean": (mean, em + E32 * mean.abs()),
        "inv_std": (inv, inv * einv)}
    if dy is None:
        return res
    g64 = dy.double()
    g = g64 * w64
    dx, dw, db = ref.layer_norm_backward(dy, x, w, eps)
    a, c = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    ea = chain * g.abs().mean(-1, keepdim=True)
    ec = chain * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * exh).mean(-1, keepdim=True)
    edx = inv[..., None] * (ea + exh * c.abs() + xh.abs() * ec + 6 * E32 * (g.abs() + a.abs() + (xh * c).abs()))
    edx = edx + dx.abs() * einv[..., None]
    res["dx"] = (dx, u * dx.abs() + (1 + u) * edx + tiny(t))
    up, chain = unit(pt), (rows + 16) * E32
    flat = (-1, n)
    ew = (g64.abs() * exh).reshape(flat).sum(0) + chain * (g64 * xh).abs().reshape(flat).sum(0)
    eb = chain * g64.abs().reshape(flat).sum(0)
    res["dscale"] = (dw, up * dw.abs() + (1 + up) * ew + tiny(pt))
    res["dbias"] = (db, up * db.abs() + (1 + up) * eb + tiny(pt))
    return res


NORMS = [(1, 1), (1, 1024), (3, 7), (2, 64), (5, 65), (7, 512), (130, 777), (33, 1000), (64, 2048), (9, 2056),
         (300, 256), (4, 4096), (3, 8192), (2, 8200), (3, 9001), (1, 20000), (1025, 24), (2049, 8)]


@pytest.mark.parametrize("rows,cols", NORMS)
@pytest.mark.parametrize("dtype,params", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_layer_norm(gs, rows, cols, dtype, params):
    t, pt = TYPES[dtype], TYPES[params]
    g = torch.Generator().manual_seed(rows * 131 + cols)
    x = (torch.randn(rows, cols, generator=g) * 1.5 + 0.7).to(t)
    w, b = (torch.randn(cols, generator=g) * 0.3 + 1).to(pt), torch.randn(cols, generator=g).to(pt)
    dy = torch.randn(rows, cols, generator=g).to(t)
    want = norm_bounds(x, w, b, dy, 1e-5, t, pt)
    X, W, B, dY = (v.cuda() for v in (x, w, b, dy))
    y, mean, inv = gs.layer_norm(X, W, B, return_stats=True)
    dx, dw, db = gs.layer_norm_backward(dY, X, W, mean, inv)
    for name, got in (("y", y), ("mean", mean), ("inv_std", inv), ("dx", dx), ("dscale", dw), ("dbias", db)):
        close(got, *want[name], name)
    assert torch.equal(gs.layer_norm(X, W, B), y)
    again = gs.layer_norm_backward(dY, X, W, mean, inv)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("rows,cols", [(70, 64), (333, 63), (40, 72), (19, 256), (21, 257), (6, 4104), (5, 8193),
                                       (3, 16385), (2, 32768), (3, 40000)])
@pytest.mark.parametrize("dtype,params", [("f32", "f32"), ("bf16", "f32")])
def test_layer_norm_of_every_form(gs, rows, cols, dtype, params):
    """Eight lanes a row up to 1024 threads, and the loops past them."""
    test_layer_norm(gs, rows, cols, dtype, params)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_layer_norm_strides_alignment_and_shapes(gs, dtype):
    """Rows apart, rows off their 16-byte alignment, a broadcast row, more axes than two, no bias."""
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(6, 5, 200, generator=g).to(t).cuda()
    w = (torch.randn(96, generator=g) + 1).to(t).cuda()
    dy = torch.randn(6, 5, 96, generator=g).to(t).cuda()
    views = {"gap": wide[..., :96], "odd": wide[..., 3:99], "row": wide[:, :1, 8:104].expand(6, 5, 96),
             "swapped": wide[..., 8:104].transpose(0, 1).contiguous().transpose(0, 1)}
    for what, x in views.items():
        want = norm_bounds(x.cpu(), w.cpu(), None, dy.cpu(), 1e-3, t, t)
        y, mean, inv = gs.layer_norm(x, w, None, 1e-3, return_stats=True)
        assert mean.shape == (6, 5)
        close(y, *want["y"], what)
        for got, name in zip(gs.layer_norm_backward(dy, x, w, mean, inv), ("dx", "dscale", "dbias")):
            close(got, *want[name], what + " " + name)


def test_layer_norm_of_constant_rows_and_nan(gs):
    """A row without variance gives its bias; a NaN stays in its row."""
    x = torch.full((3, 40), 2.5, device="cuda")
    x[1, 7] = math.nan
    w, b = torch.ones(40, device="cuda"), torch.arange(40.0, device="cuda")
    y = gs.layer_norm(x, w, b)
    assert torch.equal(y[0], b) and torch.equal(y[2], b) and y[1].isnan().all()


def test_layer_norm_without_rows(gs):
    x, w = torch.empty(0, 16, device="cuda"), torch.ones(16, device="cuda")
    y, mean, inv = gs.layer_norm(x, w, return_stats=True)
    dx, dw, db = gs.layer_norm_backward(x, x, w, mean, inv)
    assert y.shape == dx.shape == (0, 16) and not dw.any() and not db.any()


# --------------------------------------------------------------- dropout

@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 2048, 100003])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ratio,residual", [(0.0, False), (0.1, False), (0.1, True), (0.75, True)])
def test_dropout(gs, n, dtype, ratio, residual):
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g).to(t)
    r = torch.randn(n, generator=g).to(t) if residual else None
    seed = 0xFEDCBA9876543210 + n
    want = ref.dropout(x, ratio, seed, 0xFFFFFFFF, r)
    got = gs.dropout(x.cuda(), ratio, seed, 0xFFFFFFFF, None if r is None else r.cuda())
    kept = ref.dropout(x, ratio, seed, 0xFFFFFFFF).abs()
    close(got, want, unit(t) * want.abs() + 4 * E32 * (kept + want.abs()) + tiny(t), "y")


def test_dropout_layouts_in_place_and_nan(gs):
    """Off alignment, strided, in place; a dropped NaN or infinity gives 0."""
    g = torch.Generator().manual_seed(1)
    base = torch.randn(70, 91, generator=g).cuda()
    for x in (base[1:, 3:], base.t(), base.flatten()[1:]):
        want = ref.dropout(x.cpu().contiguous(), 0.3, 5, 6)
        got = gs.dropout(x, 0.3, 5, 6)
        close(got, want, 5 * E32 * want.abs(), "layout")
    x = base.clone()
    want = gs.dropout(x, 0.3, 5, 6)
    assert torch.equal(gs.dropout(x, 0.3, 5, 6, out=x), want) and torch.equal(x, want)
    bad = torch.full((4096,), math.nan, device="cuda", dtype=torch.bfloat16)
    bad[::2] = math.inf
    y, kept = gs.dropout(bad, 0.5, 3).cpu(), ref.dropout(torch.ones(4096), 0.5, 3, 0) > 0
    assert not y[~kept].any() and not y[kept].isfinite().any()


def test_dropout_gradient_is_the_same_mask(gs):
    x = torch.randn(4, 33, device="cuda") + 10
    y, dx = gs.dropout(x, 0.4, 8, 2), gs.dropout(torch.ones_like(x), 0.4, 8, 2)
    assert torch.equal(y == 0, dx == 0)


# ------------------------------------------------------------- attention

def heads(g, B, H, L, D, t, by_position):
    if by_position:
        return torch.randn(B, L, H, D, generator=g).to(t).cuda().transpose(1, 2)
    return torch.randn(B, H, L, D, generator=g).to(t).cuda()


def check_attention(gs, B, H, Hkv, Lq, Lk, D, dtype, causal=0, lengths=None, buckets=0, distance=128, both=1,
                    position=0, ratio=0.0, by_position=False, table_type=None, backward=True, seed=17):
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(B * 7 + H * 11 + Lq * 13 + Lk * 17 + D)
    q = heads(g, B, H, Lq, D, t, by_position)
    k, v = heads(g, B, Hkv, Lk, D, t, by_position), heads(g, B, Hkv, Lk, D, t, by_position)
    do = heads(g, B, H, Lq, D, t, by_position)
    table = (torch.randn(buckets, H, generator=g) * 0.7).to(TYPES[table_type or dtype]).cuda() if buckets else None
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    first = position
    if position == "end":
        n = torch.full((B,), Lk) if lens is None else lens.cpu().long().clamp(0, Lk)
        first = n - Lq
    how = dict(scale=None, causal=causal, kv_lengths=lens, table=table, max_distance=distance, bidirectional=both,
               q_position=position, ratio=ratio, seed=seed, call=9)
    cpu = lambda x: None if x is None else x.cpu()
    want = ref.attention(cpu(q), cpu(k), cpu(v), 1 / math.sqrt(D), causal, cpu(lens), cpu(table), distance, both,
                         first, ratio, seed, 9, cpu(do) if backward else None, unit(t) if t != torch.float32 else E32,
                         tiny(t))
    o, lse = gs.attention(q, k, v, return_lse=True, **how)
    assert o.stride() == q.stride() or not by_position
    close(o, *want["o"], "o")
    close(lse, *want["lse"], "lse")
    assert torch.equal(gs.attention(q, k, v, **how), o)
    if not backward:
        return
    got = gs.attention_backward(do, q, k, v, o, lse, **how)
    for name, x in zip(("dq", "dk", "dv", "dtable"), got):
        if name in want:
            close(x, *want[name], name)
    again = gs.attention_backward(do, q, k, v, o, lse, **how)
    assert all(x is None or torch.equal(x, y) for x, y in zip(got, again))


SHAPES = [  # B, H, Hkv, Lq, Lk, D
    (1, 1, 1, 1, 1, 1), (1, 1, 1, 1, 1, 64), (2, 2, 1, 3, 5, 8), (1, 4, 2, 31, 33, 16), (2, 3, 3, 64, 64, 32),
    (1, 2, 2, 65, 63, 64), (1, 2, 1, 127, 129, 64), (1, 2, 2, 128, 128, 128), (2, 4, 2, 130, 200, 40),
    (1, 5, 1, 33, 257, 63), (1, 2, 2, 129, 70, 96), (1, 3, 1, 300, 260, 80), (1, 1, 1, 5, 300, 128),
    (3, 2, 2, 17, 1, 20), (1, 1, 1, 257, 513, 64),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_plain(gs, shape, dtype):
    check_attention(gs, *shape, dtype)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_biased_dropped(gs, shape, dtype):
    check_attention(gs, *shape, dtype, buckets=32, ratio=0.2, by_position=True)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_causal(gs, shape, dtype):
    check_attention(gs, *shape, dtype, causal=1, position=shape[4] - shape[3], buckets=32, both=0, ratio=0.1)


@pytest.mark.parametrize("over", [
    dict(lengths=[0, 70, 130]), dict(lengths=[130, 1, 64], causal=1, position="end"),
    dict(lengths=[-3, 500, 65], buckets=8, distance=20), dict(causal=1, position=-40), dict(causal=1, position=-500),
    dict(causal=1, position=30, buckets=8, both=1), dict(buckets=8, both=0, distance=50),
    dict(buckets=2, both=0, distance=9), dict(buckets=320, distance=800), dict(buckets=320, distance=800, both=0),
    dict(buckets=32, distance=1000), dict(buckets=512, distance=1023, both=0, causal=1),
    dict(buckets=32, position=100), dict(buckets=32, position=-1000), dict(buckets=32, position=2 ** 29),
    dict(buckets=32, position=-(2 ** 29)), dict(ratio=0.999), dict(ratio=0.5, lengths=[0, 0, 0], buckets=4, distance=9)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_masks_and_buckets(gs, over, dtype):
    check_attention(gs, 3, 4, 2, 75, 130, 48, dtype, **over)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [0, 1])
def test_attention_table_in_fp32(gs, dtype, causal):
    check_attention(gs, 2, 4, 4, 140, 140, 64, dtype, causal=causal, buckets=32, both=1 - causal, ratio=0.1,
                    table_type="f32")


# many heads of short sequences: enough rows that blocks take 64 or 128 of them
MANY = [  # B, H, Hkv, Lq, Lk, D
    (16, 16, 16, 40, 70, 64), (32, 33, 11, 35, 65, 32), (9, 30, 15, 130, 97, 64), (37, 14, 14, 200, 131, 16),
    (4, 128, 64, 64, 64, 128), (70, 15, 5, 37, 97, 96), (5, 52, 52, 129, 257, 24), (33, 32, 32, 33, 150, 127),
]


@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("causal", [0, 1])
def test_attention_of_many_heads(gs, shape, dtype, causal):
    B, H, Hkv, Lq, Lk, D = shape
    lengths = [Lk - b * Lk // B for b in range(B)]
    lengths[-1] = 0
    check_attention(gs, *shape, dtype, causal=causal, position="end" if causal else 3, lengths=lengths, buckets=8,
                    distance=24, both=1 - causal, ratio=0.15 * causal, by_position=bool(causal))


DECODES = [(1, 8, 8, 1, 77, 64), (3, 8, 2, 1, 300, 128), (2, 8, 1, 1, 1000, 64), (1, 5, 1, 2, 2049, 40),
           (2, 4, 4, 5, 130, 63), (1, 40, 1, 1, 515, 96), (1, 12, 3, 4, 700, 32), (4, 2, 2, 1, 1, 128),
           (1, 1, 1, 1, 5000, 128), (1, 32, 4, 9, 400, 128)]


@pytest.mark.parametrize("shape", DECODES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("extras", [False, True])
def test_attention_of_few_queries(gs, shape, dtype, extras):
    B, Lk = shape[0], shape[4]
    more = dict(buckets=32, both=0, lengths=[max(0, Lk - 37 * i * i) for i in range(B)], ratio=0.1,
                by_position=True) if extras else {}
    check_attention(gs, *shape, dtype, causal=1, position="end", backward=False, **more)


def test_attention_few_queries_without_workspace(gs):
    """The same values, within rounding, when no scratch is given."""
    g = torch.Generator().manual_seed(2)
    q, k, v = (heads(g, 2, 8, n, 64, torch.float32, False) for n in (1, 3000, 3000))
    a = gs.attention(q, k, v)
    b = gs.attention(q, k, v, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    want = ref.attention(q.cpu(), k.cpu(), v.cpu(), 0.125, 0, None, None, 128, 1, 0, 0.0, 0, 0, None, E32)["o"]
    close(a, *want, "with")
    close(b, *want, "without")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_strided_inputs(gs, dtype):
    """Slices of one fused tensor, rows off alignment, broadcast heads and batch."""
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(4)
    fused = torch.randn(2, 90, 3, 4, 72, generator=g).to(t).cuda()
    def call(q, k, v, what):
        do = torch.randn(q.shape, generator=g).to(t).cuda()
        scale = 1 / math.sqrt(q.shape[-1])
        want = ref.attention(q.cpu(), k.cpu(), v.cpu(), scale, 0, None, None, 128, 1, 0, 0.0, 0, 0, do.cpu(),
                             unit(t) if t != torch.float32 else E32, tiny(t))
        o, lse = gs.attention(q, k, v, return_lse=True)
        close(o, *want["o"], what)
        for name, x in zip(("dq", "dk", "dv"), gs.attention_backward(do, q, k, v, o, lse)):
            close(x, *want[name], what + " " + name)
    def parts(lo, hi):
        return [fused[:, :, i, :, lo:hi].transpose(1, 2) for i in range(3)]
    call(*parts(0, 64), "fused")
    call(*parts(1, 65), "odd start")
    call(*parts(8, 71), "odd width")
    q, k, v = parts(0, 64)
    call(q, k[:, :1].expand(2, 4, 90, 64), v[:, :1].expand(2, 4, 90, 64), "broadcast heads")
    call(q, k[:1].expand(2, 4, 90, 64), v[:1].expand(2, 4, 90, 64), "broadcast batch")
    call(q[..., ::2], k[..., ::2], v[..., ::2], "every other element")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("Lq", [1, 70])
def test_attention_ignores_what_lies_past_a_length(gs, dtype, Lq):
    """NaN, infinities and the lowest values past the lengths change no bit; their gradients are 0."""
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(6)
    q = heads(g, 3, 2, Lq, 64, t, False)
    k, v, do = heads(g, 3, 2, 150, 64, t, False), heads(g, 3, 2, 150, 64, t, False), heads(g, 3, 2, Lq, 64, t, False)
    lens = torch.tensor([150, 67, 0], dtype=torch.int32).cuda()
    def run(fill):
        kk, vv = k.clone(), v.clone()
        for b, n in enumerate(lens.tolist()):
            kk[b, :, n:], vv[b, :, n:] = fill, fill
        o, lse = gs.attention(q, kk, vv, kv_lengths=lens, return_lse=True)
        return (o, lse) + gs.attention_backward(do, q, kk, vv, o, lse, kv_lengths=lens)[:3]
    base = run(0.0)
    for fill in (math.nan, math.inf, -math.inf, torch.finfo(t).min):
        assert all(torch.equal(a, b) for a, b in zip(base, run(fill))), fill
    assert not base[0][2].any() and (base[1][2] == -math.inf).all() and not base[2][2].any()
    assert not base[3][1, :, 67:].any() and not base[4][1, :, 67:].any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("Lk,causal", [(1, 0), (40, 1)])
def test_attention_of_one_key_has_no_gradient(gs, dtype, Lk, causal):
    """A query that sees one key: its probability is 1 whatever the scores, so its dS is 0, not a rounding."""
    g = torch.Generator().manual_seed(11)
    t = TYPES[dtype]
    q, do = heads(g, 2, 4, Lk, 48, t, False), heads(g, 2, 4, Lk, 48, t, False)
    k, v = heads(g, 2, 2, Lk, 48, t, False), heads(g, 2, 2, Lk, 48, t, False)
    how = dict(causal=causal, table=torch.randn(8, 4, generator=g).cuda(), max_distance=20, ratio=0.3, seed=2)
    o, lse = gs.attention(q, k, v, return_lse=True, **how)
    if causal:
        do[:, :, 1:] = 0
    dq, dk, dv, dt = gs.attention_backward(do, q, k, v, o, lse, **how)
    assert not dq.any() and not dk.any() and not dt.any() and dv[:, :, 0].any() and not dv[:, :, 1:].any()


def test_attention_bias_gradient_does_not_lose_what_o_rounds_off(gs):
    """Buckets that hold most keys: their sums are those of the few others, negated."""
    for dtype in ("f16", "bf16"):
        t = TYPES[dtype]
        g = torch.Generator().manual_seed(12)
        q, do = heads(g, 2, 4, 3, 32, t, False), heads(g, 2, 4, 3, 32, t, False)
        k, v = heads(g, 2, 2, 1500, 32, t, False), heads(g, 2, 2, 1500, 32, t, False)
        table = torch.randn(4, 4, generator=g).cuda()
        how = dict(table=table, max_distance=40)
        o, lse = gs.attention(q, k, v, return_lse=True, **how)
        got = gs.attention_backward(do, q, k, v, o, lse, **how)[3].cpu().double()
        want = ref.attention(q.cpu(), k.cpu(), v.cpu(), 1 / math.sqrt(32), 0, None, table.cpu(), 40, 1, 0, 0.0, 0, 0,
                             do.cpu(), unit(t), tiny(t))["dtable"][0]
        # 2^-24 for each of at most 256 roundings on the way of a dS, which is of the size of p |dO . V|
        p = torch.softmax(torch.einsum("bhid,bhjd->bhij", q.cpu().double(), k.cpu().double().repeat_interleave(2, 1)) /
                          math.sqrt(32), -1)
        size = (p * torch.einsum("bhid,bhjd->bhij", do.cpu().double(), v.cpu().double().repeat_interleave(2, 1)).abs()).sum()
        assert (got - want).abs().max() <= 2.0 ** -16 * size, dtype


def test_attention_extreme_scores(gs):
    """Scores far apart and far from zero: the softmax stays exact where one key dominates."""
    q = torch.full((1, 1, 4, 32), 30.0, device="cuda")
    k = torch.zeros(1, 1, 200, 32, device="cuda")
    k[..., 123, :] = 30.0
    k[..., 5, :] = -30.0
    v = torch.arange(200.0, device="cuda")[:, None].expand(1, 1, 200, 32).contiguous()
    o, lse = gs.attention(q, k, v, scale=1.0, return_lse=True)
    assert (o == 123).all() and (lse == 28800).all()
    o = gs.attention(q, -k, v, scale=1.0)
    assert (o == 5).all()


def test_attention_without_keys_or_queries(gs):
    q, k = torch.randn(2, 3, 4, 16, device="cuda"), torch.empty(2, 3, 0, 16, device="cuda")
    table = torch.randn(8, 3, device="cuda")
    o, lse = gs.attention(q, k, k, table=table, return_lse=True)
    assert not o.any() and (lse == -math.inf).all()
    dq, dk, dv, dt = gs.attention_backward(q, q, k, k, o, lse, table=table)
    assert not dq.any() and not dt.any() and dk.shape == dv.shape == k.shape
    e = q[:, :, :0]
    o, lse = gs.attention(e, q, q, table=table, return_lse=True)
    dq, dk, dv, dt = gs.attention_backward(e, e, q, q, o, lse, table=table)
    assert o.shape == dq.shape == e.shape and not dk.any() and not dv.any() and not dt.any()


def test_attention_backward_needs_no_table_gradient(gs):
    """Through the C entry: dtable NULL leaves dQ, dK, dV as they are with it."""
    import ctypes

    from spatial_transformer_grid_amd import _tokens as tk
    g = torch.Generator().manual_seed(8)
    q, k, v, do = (heads(g, 1, 2, 70, 32, torch.bfloat16, False) for _ in range(4))
    table = torch.randn(32, 2, generator=g).cuda()
    o, lse = gs.attention(q, k, v, table=table, return_lse=True)
    want = gs.attention_backward(do, q, k, v, o, lse, table=table)
    d = tk._attention_inputs(q, k, v, None, 0, None, table, 128, 1, 0, 0.0, 0, 0)[-1]
    got = [torch.empty_like(x) for x in (q, k, v)]
    for n in ("o", "do", "dq", "dk", "dv"):
        setattr(d, n + "_stride", tk._strides(q))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    p = tk._ptr
    st = tk.token_lib().gs_attention_backward(
        ctypes.byref(d), p(do), p(q), p(k), p(v), p(o), p(lse), None, p(table), *[p(x) for x in got], None, p(ws),
        ws.numel(), tk._stream(None, q.device))
    assert st == 0
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------- streams, graphs, errors

def test_another_stream_and_graph_replays(gs):
    """Calls on a stream of their own, then captured: every replay gives the eager bits."""
    g = torch.Generator().manual_seed(9)
    t = torch.bfloat16
    q, k, v, do = (heads(g, 2, 4, 150, 64, t, False) for _ in range(4))
    q1 = heads(g, 2, 4, 1, 64, t, False)
    table, x = torch.randn(32, 4, generator=g).to(t).cuda(), torch.randn(130, 264, generator=g).to(t).cuda()
    w = torch.ones(264, device="cuda", dtype=t)

    def step():
        y, mean, inv = gs.layer_norm(x, w, w, return_stats=True)
        z = gs.dropout(y, 0.1, 1, residual=x)
        grads = gs.layer_norm_backward(z, x, w, mean, inv)
        how = dict(table=table, ratio=0.1, seed=4)
        o, lse = gs.attention(q, k, v, return_lse=True, **how)
        return (y, z, o, gs.attention(q1, k, v, table=table)) + grads + gs.attention_backward(do, q, k, v, o, lse, **how)

    eager = [a.clone() for a in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        own = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, own))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        for a in held:
            a.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held))
        assert all(torch.equal(a, b) for a, b in zip(eager, step()))


def test_binding_refusals(gs):
    q = torch.zeros(2, 4, 5, 16, device="cuda")
    for bad in [lambda: gs.attention(q, q[:1], q[:1]), lambda: gs.attention(q, q, q[..., :3, :]),
                lambda: gs.attention(q, q, q, kv_lengths=torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: gs.attention(q, q, q, table=torch.zeros(8, 3, device="cuda")),
                lambda: gs.attention(q, q, q, table=torch.zeros(1, 4, device="cuda")),
                lambda: gs.attention(q, q, q, q_position="start"),
                lambda: gs.attention(q, q, q, out=q[..., :8]),
                lambda: gs.attention_backward(q, q, q, q, q, q[..., 0, 0]),
                lambda: gs.layer_norm(q, q[0, 0, 0, :8]), lambda: gs.dropout(q, 0.1, 1, residual=q[:1])]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: gs.attention(q, q.half(), q), lambda: gs.attention(q, q, q.half()),
                lambda: gs.attention(q, q, q, kv_lengths=torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: gs.attention(q.half(), q.half(), q.half(), table=torch.zeros(8, 4, device="cuda").bfloat16()),
                lambda: gs.layer_norm(q.half(), q[0, 0, 0].bfloat16())]:
        with pytest.raises(TypeError):
            bad()
    for bad, status in [(lambda: gs.attention(q, q[:, :3], q[:, :3]), 2), (lambda: gs.dropout(q, 1.0, 1), 4),
                        (lambda: gs.attention(q, q, q, ratio=-0.5), 4), (lambda: gs.attention(q, q, q, causal=2), 4),
                        (lambda: gs.layer_norm(q, q[0, 0, 0], epsilon=-1.0), 4)]:
        with pytest.raises(gs.GSError) as e:
            bad()
        assert e.value.status == status
    with pytest.raises(gs.GSError):
        big = torch.zeros(1, 1, 2, 136, device="cuda")
        gs.attention(big, big, big)
