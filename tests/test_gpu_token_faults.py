"""The token operators on the GPU where a value, a layout or a stream is out of
the ordinary: NaN and masks of the lowest values, streams given by name, forms
that only large grids take, tensors past 2^31 elements.  Bounds are
token_reference's."""

import math

import pytest
import torch

import token_reference as ref
from test_gpu_tokens import E32, TYPES, check_attention, close, heads, tiny, unit

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import spatial_transformer_grid_amd as gs

    gs.token_lib()
    return gs


# ------------------------------------------------------------------- NaN

FORMS = {  # B, H, Hkv, Lq, Lk: the row form, the split of the keys and the packing that they take
    "128 rows": (16, 16, 16, 200, 70), "32 rows": (1, 2, 2, 40, 200), "split": (1, 8, 8, 1, 3000),
    "packed": (3, 8, 2, 1, 200), "packed and split": (1, 8, 2, 3, 3000)}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ratio", [0.0, 0.3])
def test_attention_nan_query_gives_nan(gs, form, dtype, ratio):
    """A NaN in a query reaches its whole output row and its lse in every form, and no other row."""
    B, H, Hkv, Lq, Lk = FORMS[form]
    g = torch.Generator().manual_seed(1)
    t = TYPES[dtype]
    q, k, v = (heads(g, B, n, length, 64, t, False) for n, length in ((H, Lq), (Hkv, Lk), (Hkv, Lk)))
    how = dict(return_lse=True, table=torch.randn(8, H, generator=g).to(t).cuda(), max_distance=20, ratio=ratio, seed=3)
    o, lse = gs.attention(q, k, v, **how)
    q[0, 1, Lq - 1, 5] = math.nan
    got, got_lse = gs.attention(q, k, v, **how)
    assert got[0, 1, Lq - 1].isnan().all() and got_lse[0, 1, Lq - 1].isnan()
    got[0, 1, Lq - 1], got_lse[0, 1, Lq - 1] = o[0, 1, Lq - 1], lse[0, 1, Lq - 1]
    assert torch.equal(got, o) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_nan_key_reaches_the_queries_that_see_it(gs, form, dtype):
    """A NaN in a key's row, the last one, seen by the last query alone."""
    B, H, Hkv, Lq, Lk = FORMS[form]
    g = torch.Generator().manual_seed(2)
    t = TYPES[dtype]
    q, k, v = (heads(g, B, n, length, 64, t, False) for n, length in ((H, Lq), (Hkv, Lk), (Hkv, Lk)))
    how = dict(return_lse=True, causal=1, q_position=Lk - Lq)
    o, lse = gs.attention(q, k, v, **how)
    k[0, 0, Lk - 1, 7] = math.nan
    got, got_lse = gs.attention(q, k, v, **how)
    G = H // Hkv
    assert got[0, :G, Lq - 1].isnan().all() and got_lse[0, :G, Lq - 1].isnan().all()
    got[0, :G, Lq - 1], got_lse[0, :G, Lq - 1] = o[0, :G, Lq - 1], lse[0, :G, Lq - 1]
    assert torch.equal(got, o) and torch.equal(got_lse, lse)


# ------------------------------------------------- keys without query heads

@pytest.mark.parametrize("Lk", [7, 300])
@pytest.mark.parametrize("table", [False, True])
def test_attention_gradients_without_query_heads_are_zero(gs, Lk, table):
    q, k = torch.empty(2, 0, 5, 24, device="cuda"), torch.randn(2, 4, Lk, 24, device="cuda")
    used = [torch.full_like(k, 7.0) for _ in range(6)]
    del used                                         # what a new tensor is likely to hold
    how = dict(table=torch.empty(8, 0, device="cuda")) if table else {}
    o, lse = gs.attention(q, k, k, return_lse=True, **how)
    dq, dk, dv, _ = gs.attention_backward(q, q, k, k, o, lse, **how)
    assert dq.shape == q.shape and dk.shape == dv.shape == k.shape and not dk.any() and not dv.any()


# ---------------------------------------------------------------- streams

def test_calls_on_a_stream_given_by_name(gs):
    """stream=s with strided inputs that the current stream has only just been asked to write, s busy, and the current
    stream's allocations filled right after each call: the bits are those of plain calls."""
    g = torch.Generator().manual_seed(21)
    t = torch.bfloat16
    wide = torch.randn(2, 300, 4, 128, generator=g).to(t).cuda()
    rows = torch.randn(600, 2 * 264, generator=g).to(t).cuda()
    q1 = torch.randn(2, 1, 4, 128, generator=g).to(t).cuda()
    table = torch.randn(4, 32, generator=g).to(t).cuda()
    square = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()

    def busy(n):
        for _ in range(n):
            torch.mm(square, square)

    def calls(stream):
        """Every call's outputs; the inputs are made anew and die at once."""
        def every_other(x):
            return (x * 1.0)[..., ::2]               # its last axis is copied by the call
        def heads_of(x):
            return every_other(x).transpose(1, 2)
        def after():
            if stream is not None:
                for n in (1 << 10, 1 << 16, 1 << 20, 1 << 24):
                    for _ in range(4):
                        torch.full((n,), float("nan"), device="cuda")
        out = []
        x, w = every_other(rows), torch.ones(264, device="cuda", dtype=t)
        y, mean, inv = gs.layer_norm(x, w, w, return_stats=True, stream=stream)
        after()
        out += [y, mean, inv, *gs.layer_norm_backward(every_other(rows) + 1, x, w, mean, inv, stream=stream)]
        after()
        out.append(gs.dropout(every_other(rows), 0.2, 7, residual=x, stream=stream))
        after()
        how = dict(table=table.t() * 1.0, ratio=0.1, seed=5, stream=stream)
        o, lse = gs.attention(heads_of(wide), heads_of(wide) + 1, heads_of(wide) * 2, return_lse=True, **how)
        after()
        out += [o, lse, *gs.attention_backward(heads_of(wide) - 1, heads_of(wide), heads_of(wide) + 1, heads_of(wide) * 2,
                                               o, lse, **how)]
        after()
        out.append(gs.attention(heads_of(q1), heads_of(wide), heads_of(wide), stream=stream))
        after()
        return out

    want = calls(None)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream, torch.cuda.current_stream(), 0):
        busy(3)
        with torch.cuda.stream(s):
            busy(6)
        got = calls(stream)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()


def test_older_calls_on_a_stream_given_by_name(gs):
    """The sampler, Resize and DeformConv with its scratch, the same way."""
    g = torch.Generator().manual_seed(22)
    X = torch.randn(2, 16, 24, 2 * 24, generator=g).cuda()
    W = torch.randn(16, 16, 3, 3, generator=g).cuda()
    offset = torch.randn(2, 18, 24, 24, generator=g).cuda()
    theta = torch.eye(2, 3).repeat(2, 1, 1).cuda() * 0.9
    square = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()

    def calls(stream):
        x = lambda: (X * 1.0)[..., ::2]
        out = [gs.affine_grid(theta * 1.0, (2, 16, 24, 24), stream=stream)]
        out.append(gs.grid_sample(x(), out[0] * 1.0 if stream is None else out[0], workspace="auto", stream=stream))
        out.append(gs.affine_grid_sample_fused(theta * 1.0, x(), (24, 24), stream=stream))
        out.append(gs.resize(x(), sizes=(2, 16, 48, 40), mode="linear", stream=stream))
        out.append(gs.resize_to(x(), (2, 16, 48, 40), mode="linear", stream=stream))
        out.append(gs.deform_conv(x(), W * 1.0, offset * 1.0, pads=[1, 1, 1, 1], stream=stream))
        if stream is not None:
            for n in (1 << 12, 1 << 20, 1 << 22):
                torch.full((n,), float("nan"), device="cuda")
        return out

    want = calls(None)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        for _ in range(3):
            torch.mm(square, square)
        got = calls(stream)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()


def test_calls_on_a_named_stream_captured(gs):
    """A branch of a captured graph: calls with stream=s between the fork that they make and the caller's join."""
    g = torch.Generator().manual_seed(23)
    t = torch.float16
    q, k, v, do = (heads(g, 2, 4, 150, 64, t, True) for _ in range(4))
    q1, table = heads(g, 2, 4, 1, 64, t, True), torch.randn(32, 4, generator=g).to(t).cuda()
    x, w = torch.randn(130, 2 * 264, generator=g).to(t).cuda(), torch.ones(264, device="cuda", dtype=t)
    s = torch.cuda.Stream()

    def step(stream):
        rows = x[:, ::2]
        y, mean, inv = gs.layer_norm(rows, w, w, return_stats=True, stream=stream)
        grads = gs.layer_norm_backward(y, rows, w, mean, inv, stream=stream)
        how = dict(table=table, ratio=0.1, seed=4, stream=stream)
        o, lse = gs.attention(q, k, v, return_lse=True, **how)
        one = gs.attention(q1, k, v, stream=stream)
        return [y, o, lse, one, *grads, *gs.attention_backward(do, q, k, v, o, lse, **how)]

    eager = [a.clone() for a in step(None)]
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for a in held:
            a.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held))
        assert all(torch.equal(a, b) for a, b in zip(eager, step(None)))


# --------------------------------------------------------------- refusals

def test_scratch_in_host_memory_is_refused(gs):
    x, w = torch.randn(4, 16, device="cuda"), torch.ones(16, device="cuda")
    q = torch.randn(1, 2, 40, 16, device="cuda")
    y, mean, inv = gs.layer_norm(x, w, return_stats=True)
    o, lse = gs.attention(q, q, q, return_lse=True)
    image, kernel = torch.randn(1, 4, 8, 8, device="cuda"), torch.randn(4, 4, 3, 3, device="cuda")
    offset, grid = torch.zeros(1, 18, 6, 6, device="cuda"), torch.zeros(1, 6, 6, 2, device="cuda")
    for bad in (torch.empty(1 << 16, dtype=torch.uint8), torch.empty(1 << 17, dtype=torch.uint8, device="cuda")[::2]):
        for call in (lambda: gs.layer_norm_backward(x, x, w, mean, inv, workspace=bad),
                     lambda: gs.attention(q, q, q, workspace=bad),
                     lambda: gs.attention_backward(q, q, q, q, o, lse, workspace=bad),
                     lambda: gs.deform_conv(image, kernel, offset, workspace=bad),
                     lambda: gs.grid_sample(image, grid, workspace=bad)):
            with pytest.raises(ValueError):
                call()


def test_attention_refuses_an_expanded_output(gs):
    q = torch.randn(2, 3, 5, 16, device="cuda")
    for out in (torch.empty(2, 3, 1, 16, device="cuda").expand(2, 3, 5, 16),
                torch.empty(1, 3, 5, 16, device="cuda").expand(2, 3, 5, 16),
                torch.empty(2, 3, 200, device="cuda").as_strided((2, 3, 5, 16), (600, 200, 8, 1))):
        with pytest.raises(gs.GSError) as e:
            gs.attention(q, q, q, out=out)
        assert e.value.status == 2


# ---------------------------------------------------------- launch limits

def test_attention_of_as_many_blocks_as_a_launch_takes(gs):
    for heads_, ok in ((2 ** 20 - 1, True), (2 ** 20, False)):
        q = torch.ones(16, heads_, 1, 1, device="cuda", dtype=torch.float16)
        if ok:
            o, lse = gs.attention(q, q, q, return_lse=True)
            assert (o == 1).all() and (lse == 1).all()
        else:
            with pytest.raises(gs.GSError) as e:
                gs.attention(q, q, q)
            assert e.value.status == 6
    q = torch.ones(1, 2 ** 14, 1, 1, device="cuda", dtype=torch.float16)
    table = torch.zeros(512, 2 ** 14, device="cuda", dtype=torch.float16)
    how = dict(table=table, max_distance=1000)
    o, lse = gs.attention(q, q, q, return_lse=True, **how)
    assert not gs.attention_backward(q, q, q, q, o, lse, **how)[3].any()


# ------------------------------------------------------------------- norm

@pytest.mark.parametrize("cols", [1, 3, 8, 10, 40, 72, 100, 264, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_backward_of_large_constant_rows(gs, cols, dtype):
    """A row of one large value (without variance; mean * inv_std passes the largest fp32) has xh = 0, so that
    dx = inv_std (g - mean(g)) and dscale = 0; other rows are as without it."""
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(5, cols, generator=g).to(t)
    x[2] = 2.0 ** 118                                # its sum of up to 300 columns stays finite
    dy = torch.randn(5, cols, generator=g).to(t)
    w = (torch.randn(cols, generator=g) + 1).to(t)
    X, dY, W = x.cuda(), dy.cuda(), w.cuda()
    y, mean, inv = gs.layer_norm(X, W, return_stats=True)
    assert not y[2].any() and mean[2] == 2.0 ** 118
    dx, dw, db = gs.layer_norm_backward(dY, X, W, mean, inv)
    gw = dy[2].double() * w.double()
    want = (gw - gw.mean()) / math.sqrt(1e-5)
    # g, its mean (a sum of `cols` terms), the difference and inv_std round once or twice each
    bound = unit(t) * want.abs() + 1.01 * ((cols + 8) * E32 * (gw.abs() + gw.abs().mean()) / math.sqrt(1e-5))
    close(dx[2], want, bound, "dx")
    rest = [0, 1, 3, 4]
    alone = gs.layer_norm_backward(dY[rest], X[rest], W, mean[rest], inv[rest])
    assert torch.equal(dx[rest], alone[0])
    ref_w = ref.layer_norm_backward(dy[rest], x[rest], w, 1e-5)[1]
    close(dw, ref_w, unit(t) * ref_w.abs() + 1e-3 * dy.double().abs().sum(0), "dscale")


@pytest.mark.parametrize("cols", [41, 47, 82, 328, 656, 1128, 2256, 4512, 8437, 9024, 17704, 33255])
@pytest.mark.parametrize("value", [1.0, 2.5, -1e4])
def test_layer_norm_of_constant_rows_is_the_bias(gs, cols, value):
    """Widths whose rounded reciprocal is not good enough for a mean: a sum that is exact has an exact mean."""
    x, w = torch.full((3, cols), value, device="cuda"), torch.ones(cols, device="cuda")
    b = torch.arange(float(cols), device="cuda")
    y, mean, inv = gs.layer_norm(x, w, b, return_stats=True)
    assert (mean == value).all() and torch.equal(y, b.expand(3, cols))


# --------------------------------------------- forms of large grids alone

@pytest.mark.parametrize("shape", [(4, 64, 16, 520, 33, 64), (4, 32, 8, 520, 201, 128), (2, 64, 32, 1100, 77, 48),
                                   (8, 8, 8, 1030, 65, 128)])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("over", [dict(buckets=8, distance=24, ratio=0.2),
                                  dict(causal=1, position="end", ragged=True, by_position=True),
                                  dict(causal=1, position=-3, buckets=32, both=0, ratio=0.1, ragged=True)])
def test_attention_backward_of_split_128_key_blocks(gs, shape, dtype, over):
    """dK / dV blocks of 128 keys whose queries are split over parts, a part from the middle of a head on."""
    over = dict(over)
    if over.pop("ragged", False):
        B, Lk = shape[0], shape[4]
        over["lengths"] = [Lk - b * Lk // B for b in range(B - 1)] + [0]
    check_attention(gs, *shape, dtype, **over)


# ------------------------------------------------------------ small scratch

def test_attention_with_less_scratch_than_it_asks_for(gs):
    """Scratch that is too small for a split of the keys is left alone, and the call is as without any."""
    g = torch.Generator().manual_seed(31)
    q, k, v = (heads(g, 1, 8, n, 64, torch.bfloat16, False) for n in (1, 3000, 3000))
    none = gs.attention(q, k, v, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    small = torch.full((256,), 7, dtype=torch.uint8, device="cuda")
    assert torch.equal(gs.attention(q, k, v, workspace=small), none) and (small == 7).all()


# ----------------------------------------------- past 2^31 elements or bytes

@pytest.mark.parametrize("step", [1 << 22, (1 << 22) + 8, (1 << 22) + 1])
def test_attention_of_rows_far_apart(gs, step):
    """A cache whose rows lie up to 2^31.5 elements from its first, queries as far: the bits of dense tensors."""
    g = torch.Generator().manual_seed(32)
    t = torch.bfloat16
    n = 700
    cache = torch.empty(n * step + 512, dtype=t, device="cuda")
    far = lambda at, heads_, length, s: cache.as_strided((1, heads_, length, 64), (n * step, 64, s, 1), at)
    dense = [heads(g, 1, h, length, 64, t, False) for h, length in ((4, 65), (2, n), (2, n), (4, 65))]
    views = [far(256, 4, 65, 10 * step), far(0, 2, n, step), far(128, 2, n, step)]
    for view, x in zip(views, dense):
        view.copy_(x)
    how = dict(table=torch.randn(8, 4, generator=g).to(t).cuda(), max_distance=20, causal=1, q_position=n - 65)
    o, lse = gs.attention(*views, out=torch.empty_like(dense[0]), return_lse=True, **how)
    want, want_lse = gs.attention(*dense[:3], return_lse=True, **how)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert torch.equal(gs.attention(views[0][:, :, -1:], *views[1:], **{**how, "q_position": n - 1}),
                       gs.attention(dense[0][:, :, -1:], *dense[1:3], **{**how, "q_position": n - 1}))
    got = gs.attention_backward(dense[3], *views, o, lse, **how)
    for a, b in zip(got, gs.attention_backward(dense[3], *dense[:3], o, lse, **how)):
        assert torch.equal(a, b)


def test_layer_norm_past_2_31_elements(gs):
    t = torch.bfloat16
    w = torch.ones(1032, device="cuda", dtype=t)
    rows = (1 << 21) + 3
    x = torch.empty(rows, 1032, device="cuda", dtype=t)
    x[:-4096].fill_(1.0)
    x[-4096:] = torch.randn(4096, 1032, device="cuda", dtype=t)
    y, mean, inv = gs.layer_norm(x, w, return_stats=True)
    tail = gs.layer_norm(x[-4096:], w, return_stats=True)
    assert torch.equal(y[-4096:], tail[0]) and torch.equal(mean[-4096:], tail[1]) and torch.equal(inv[-4096:], tail[2])
    assert not y[:64].any()
    del tail
    dx = gs.layer_norm_backward(y, x, w, mean, inv)[0]
    assert torch.equal(dx[-4096:], gs.layer_norm_backward(y[-4096:], x[-4096:], w, mean[-4096:], inv[-4096:])[0])
    del y, dx
    apart = x.flatten().as_strided((3, 1032), (1 << 30, 1))
    assert torch.equal(gs.layer_norm(apart, w), gs.layer_norm(apart.clone(), w))


def test_dropout_past_2_31_elements(gs):
    import numpy as np

    n, first = (1 << 31) + 100003, (1 << 31) - 4096
    x = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    y = gs.dropout(x, 0.3, 11, 2)[first:].cpu()
    at = np.arange(first // 8, (n + 7) // 8, dtype=np.uint64)
    want = ref.factors(ref.numbers((at, 0, 0, 2), 11).reshape(-1)[:n - first], 0.3)
    close(y, want, unit(torch.bfloat16) * want + 4 * E32 * want, "y")


# ------------------------------------------- tables that mask by large values

MASKS = {"-1e4": -1e4, "f16 lowest": -65504.0, "-1e6": -1e6, "-1e9": -1e9, "lowest": None, "1e9": 1e9}
MASKED = {  # which buckets of 8 (both sides) hold the mask, and a shape with lengths: queries that see no other key
    "far before": ([2, 3], (2, 4, 2, 150, 150, 32), [20, 150]), "everywhere": (list(range(8)), (1, 2, 2, 40, 300, 64), None),
    "after": ([4, 5, 6, 7], (2, 2, 1, 70, 33, 48), [33, 5]), "many": ([2, 3], (9, 30, 15, 130, 97, 64), None),
    "few queries": ([2, 3, 7], (1, 8, 2, 3, 1500, 64), None)}


@pytest.mark.parametrize("mask,dtype,table_type", [
    (m, *types) for m, v in MASKS.items() for types in (("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"))
    if types[1] != "f16" or v is None or abs(v) <= 65504])
@pytest.mark.parametrize("where", list(MASKED))
@pytest.mark.parametrize("ratio", [0.0, 0.2])
def test_attention_of_tables_that_mask(gs, mask, where, dtype, table_type, ratio):
    """A constant leaves the softmax as it is, so a query that sees masked keys alone has the one of the products, and
    the others have none of a masked key.  The oracle's mask is -300 (for 1e9: 300), whose e^-300 stands for 0."""
    buckets, (B, H, Hkv, Lq, Lk, D), lengths = MASKED[where]
    t, tt = TYPES[dtype], TYPES[table_type]
    value = torch.finfo(tt).min if MASKS[mask] is None else MASKS[mask]
    g = torch.Generator().manual_seed(41)
    q, do = heads(g, B, H, Lq, D, t, True), heads(g, B, H, Lq, D, t, True)
    k, v = heads(g, B, Hkv, Lk, D, t, True), heads(g, B, Hkv, Lk, D, t, True)
    q *= 3                                           # products of up to about 40 in base 2
    table = torch.randn(8, H, generator=g).to(tt)
    like = table.clone()
    table[buckets], like[buckets] = value, math.copysign(300.0, value)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    how = dict(table=table.cuda(), max_distance=20, kv_lengths=None if lens is None else lens.cuda(), ratio=ratio, seed=3)
    first = -Lq if where == "after" else 0           # there all keys are after the queries
    want = ref.attention(q.cpu(), k.cpu(), v.cpu(), 1 / math.sqrt(D), 0, lens, like, 20, 1, first, ratio, 3, 0,
                         do.cpu(), unit(t) if t != torch.float32 else E32, tiny(t))
    want = {n: (torch.where(x.abs() < 1e-100, 0.0, x), e) for n, (x, e) in want.items()}
    o, lse = gs.attention(q, k, v, return_lse=True, q_position=first, **how)
    close(o, *want["o"], "o")
    natural = want["lse"][0]
    alone = natural < -150 if value < 0 else natural > 150
    assert alone.any() or where == "few queries"
    kept = ~alone & (natural > -math.inf)
    close(lse.cpu()[kept], natural[kept], want["lse"][1][kept], "lse")
    assert ((lse.cpu()[alone] - value).abs() <= 1e-2 * abs(value)).all()
    assert torch.equal(lse.cpu() == -math.inf, natural == -math.inf)
    got = gs.attention_backward(do, q, k, v, o, lse, q_position=first, **how)
    for name, x in zip(("dq", "dk", "dv", "dtable"), got):
        close(x, *want[name], name)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_of_an_infinite_mask_hides_its_keys(gs, dtype):
    """-inf in the table: a query left without keys gives 0 and lse -inf, and no gradient."""
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(42)
    q, k, v, do = (heads(g, 2, 2, 150, 32, t, False) for _ in range(4))
    table = torch.randn(8, 2, generator=g).to(t)
    table[2:4] = -math.inf                           # of keys 10 and more before the query, and no others
    lens = torch.tensor([20, 150], dtype=torch.int32)
    how = dict(table=table.cuda(), max_distance=20, kv_lengths=lens.cuda())
    like = table.clone()
    like[2:4] = -300.0
    none = ref.bucket(torch.arange(150).numpy()[None] - torch.arange(150).numpy()[:, None], 8, 20, 1)
    none = torch.from_numpy(((none == 2) | (none == 3))[:, :20].all(1))
    assert none.any()
    do[0, :, none.cuda()] = 0
    want = ref.attention(q.cpu(), k.cpu(), v.cpu(), 1 / math.sqrt(32), 0, lens, like, 20, 1, 0, 0.0, 0, 0, do.cpu(),
                         unit(t) if t != torch.float32 else E32, tiny(t))
    want = {n: (torch.where(x.abs() < 1e-100, 0.0, x), e) for n, (x, e) in want.items()}
    o, lse = gs.attention(q, k, v, return_lse=True, **how)
    assert not o[0, :, none.cuda()].any() and (lse[0, :, none.cuda()] == -math.inf).all()
    got = gs.attention_backward(do, q, k, v, o, lse, **how)
    assert not got[0][0, :, none.cuda()].any()
    for x in (o, got[0]):
        x[0, :, none.cuda()] = 0
    for name, x in zip(("o", "dq", "dk", "dv", "dtable"), (o, *got)):
        value, bound = want[name]
        if name == "o":
            value[0, :, none] = 0
        if name == "dq":
            value[0, :, none] = 0
        close(x, value, bound, name)


# ------------------------------------------------- queries that see no key

@pytest.mark.parametrize("shape", [(2, 4, 2, 64, 150, 64), (16, 16, 16, 200, 70, 64), (1, 2, 1, 300, 40, 48),
                                   (64, 8, 8, 170, 130, 128), (4, 64, 16, 520, 33, 63)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_queries_before_the_first_token_may_hold_nan(gs, shape, dtype):
    """More queries than a sequence has tokens (padding before them): what Q and dO hold there reaches no gradient."""
    B, H, Hkv, Lq, Lk, D = shape
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(51)
    q, do = heads(g, B, H, Lq, D, t, True), heads(g, B, H, Lq, D, t, True)
    k, v = heads(g, B, Hkv, Lk, D, t, True), heads(g, B, Hkv, Lk, D, t, True)
    lens = torch.tensor([max(0, min(Lk, Lq) - 1 - 9 * b) for b in range(B)], dtype=torch.int32)
    how = dict(causal=1, q_position="end", kv_lengths=lens.cuda(), table=torch.randn(8, H, generator=g).to(t).cuda(),
               max_distance=20, bidirectional=0, ratio=0.1, seed=2)
    def run(fill):
        a, d = q.clone(), do.clone()
        for b, n in enumerate(lens.tolist()):
            a[b, :, :Lq - n], d[b, :, :Lq - n] = fill, fill
        o, lse = gs.attention(a, k, v, return_lse=True, **how)
        return (o, lse) + gs.attention_backward(d, a, k, v, o, lse, **how)
    base = run(0.0)
    assert all(x.isfinite().all() for x in base[2:]) and not base[0][0, :, :Lq - lens[0]].any()
    assert not base[2][0, :, :Lq - lens[0]].any()
    for fill in (math.nan, math.inf):
        assert all(torch.equal(a, b) for a, b in zip(base, run(fill))), fill


# -------------------------------------------- gradients under heavy dropout

@pytest.mark.parametrize("shape", [(1, 15, 3, 239, 239, 1), (18, 5, 1, 89, 277, 1), (8, 6, 3, 1, 480, 3),
                                   (24, 16, 16, 1, 240, 64), (64, 16, 16, 130, 140, 2)])
@pytest.mark.parametrize("dtype,ratio", [("f16", 0.9), ("f16", 0.5), ("f16", 0.9999), ("bf16", 0.9), ("f32", 0.9999)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_attention_gradients_of_small_numbers_under_dropout(gs, shape, dtype, ratio, seed):
    """Scores' gradients near fp16's smallest normal value are rounded as they are, keep_scale included."""
    check_attention(gs, *shape, dtype, ratio=ratio, buckets=8, distance=9, both=0, seed=seed)
