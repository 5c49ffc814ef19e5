"""The gated projections, the norms around a block and the gated recurrence on
the GPU against the 64-bit reference, at the sizes, layouts and masks where they
can go wrong.  Every bound is derived from the roundings a kernel makes
(block_reference), none from a run."""

import math

import pytest
import torch

import block_reference as ref
from test_gpu_tokens import TYPES, close

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def gs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import spatial_transformer_grid_amd as gs

    gs.token_lib()
    return gs


def maker(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, scale=1.0, mean=0.0, t=torch.float32: (torch.randn(*s, generator=g) * scale + mean).to(t)


# ------------------------------------------------------- gated projections

def check_gated(gs, x, wg, wu, act, dy, X=None, dY=None):
    want = ref.gated(x, wg, wu, act, dy)
    X = x.cuda() if X is None else X
    WG, WU = wg.cuda(), wu.cuda()
    y = gs.gated_linear(X, WG, WU, act)
    close(y, *want["y"], "y")
    if dy is None:
        return
    dY = dy.cuda() if dY is None else dY
    again, saved = gs.gated_linear(X, WG, WU, act, return_saved=True)
    assert torch.equal(again, y)
    close(saved[0], *want["a"], "a")
    close(saved[1], *want["b"], "b")
    got = gs.gated_linear_backward(dY, X, WG, WU, saved, act)
    for name, v in zip(("dx", "dgate", "dup"), got):
        close(v, *want[name], name)
    assert all(torch.equal(p, q) for p, q in zip(got, gs.gated_linear_backward(dY, X, WG, WU, saved, act)))


GATED = [(1, 1, 1), (1, 8, 16), (1, 1000, 24), (2, 33, 17), (16, 64, 64), (17, 40, 100), (33, 72, 136), (64, 520, 31),
         (65, 64, 64), (65, 7, 300), (130, 130, 130), (200, 257, 9), (257, 96, 129), (500, 33, 250), (3, 2049, 5),
         (70, 1500, 40), (1000, 8, 8), (1300, 24, 40), (2, 5, 2000)]


@pytest.mark.parametrize("rows,width,hidden", GATED)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gated_linear(gs, rows, width, hidden, dtype):
    t, r = TYPES[dtype], maker(rows * 7 + width * 3 + hidden)
    act = ACTS[(rows + width + hidden) % 4]
    check_gated(gs, r(rows, width, t=t), r(hidden, width, scale=width ** -0.5, t=t),
                r(hidden, width, scale=width ** -0.5, t=t), act, r(rows, hidden, t=t))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gated_linear_activations(gs, act, dtype):
    """Projections from -40 to 40, where an activation ends in 0 or in its argument."""
    t, r = TYPES[dtype], maker(3)
    check_gated(gs, r(70, 16, scale=3.0, t=t), r(90, 16, t=t), r(90, 16, t=t), act, r(70, 90, t=t))


@pytest.mark.parametrize("rows,width,hidden", [(3500, 264, 2100), (260, 4096, 264), (2100, 520, 4200)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gated_linear_of_large_tiles_and_long_sums(gs, rows, width, hidden, dtype):
    t, r = TYPES[dtype], maker(rows)
    check_gated(gs, r(rows, width, t=t), r(hidden, width, scale=width ** -0.5, t=t),
                r(hidden, width, scale=width ** -0.5, t=t), "silu", r(rows, hidden, t=t))


@pytest.mark.parametrize("rows", [5, 150])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gated_linear_strides_alignment_and_shapes(gs, rows, dtype):
    """Rows apart, rows off their alignment, a broadcast row, more axes than two, weights off their alignment."""
    t, r = TYPES[dtype], maker(8)
    wide, dwide = r(rows, 2, 200, t=t), r(rows, 2, 300, t=t)
    buffer = r(2 * 80 * 96 + 3, t=t).cuda()
    for first, lo in ((0, 0), (3, 3), (2, 2), (1, 8)):
        wg, wu = (buffer[first + i * 80 * 96:][:80 * 96].view(80, 96) for i in range(2))
        for x in (wide[..., lo:lo + 96], wide[:, :1, lo:lo + 96].expand(rows, 2, 96)):
            dy = dwide[..., lo:lo + 80]
            gpu = wide.cuda()[..., lo:lo + 96] if x.stride(1) else wide.cuda()[:, :1, lo:lo + 96].expand(rows, 2, 96)
            want = ref.gated(x.reshape(-1, 96), wg.cpu(), wu.cpu(), "gelu", dy.reshape(-1, 80))
            y, saved = gs.gated_linear(gpu, wg, wu, "gelu", return_saved=True)
            assert y.shape == (rows, 2, 80) and saved.shape == (2, rows, 2, 80)
            close(y.reshape(-1, 80), *want["y"], "y")
            got = gs.gated_linear_backward(dwide.cuda()[..., lo:lo + 80], gpu, wg, wu, saved, "gelu")
            assert got[0].shape == (rows, 2, 96)
            for name, v in zip(("dx", "dgate", "dup"), got):
                close(v.reshape(want[name][0].shape), *want[name], name)


def test_gated_linear_without_rows_or_units(gs):
    w = torch.randn(6, 8, device="cuda")
    y, saved = gs.gated_linear(torch.empty(0, 8, device="cuda"), w, w, return_saved=True)
    assert y.shape == (0, 6) and saved.shape == (2, 0, 6)
    used = torch.full((6, 8), 7.0, device="cuda")
    del used                                         # what a new tensor is likely to hold
    dx, dg, du = gs.gated_linear_backward(y, torch.empty(0, 8, device="cuda"), w, w, saved)
    assert dx.shape == (0, 8) and not dg.any() and not du.any()
    x, none = torch.randn(5, 8, device="cuda"), w[:0]
    y, saved = gs.gated_linear(x, none, none, return_saved=True)
    assert y.shape == (5, 0)
    dx, dg, _ = gs.gated_linear_backward(y, x, none, none, saved)
    assert not dx.any() and dx.shape == x.shape and dg.shape == (0, 8)


@pytest.mark.parametrize("rows", [4, 40, 300])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gated_linear_nan_and_infinities_stay_in_their_rows(gs, rows, dtype):
    t, r = TYPES[dtype], maker(4)
    x, w, u = r(rows, 72, t=t).cuda(), r(90, 72, t=t).cuda(), r(90, 72, t=t).cuda()
    y = gs.gated_linear(x, w, u)
    bad = x.clone()
    bad[1, 5], bad[2, 71] = math.nan, math.inf
    got = gs.gated_linear(bad, w, u)
    assert got[1].isnan().all() and not got[2].isfinite().all()
    assert torch.equal(got[3:], y[3:]) and torch.equal(got[0], y[0])
    w[7, 3] = math.nan
    got = gs.gated_linear(x, w, u)
    assert got[:, 7].isnan().all()
    got[:, 7] = y[:, 7]
    assert torch.equal(got, y)


# --------------------------------------------------- norms around a block

def check_join(gs, x, branch, how, train=True, gpu=None):
    """`how`: post, post_bias, pre, pre_bias, gate, alpha, norm, dh, dy on the CPU."""
    c = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in how.items()}
    X, F = (x.cuda(), branch.cuda()) if gpu is None else gpu
    want = ref.join(x, branch, how["post"], how["post_bias"], how["pre"], how["pre_bias"], how["gate"], how["alpha"],
                    1e-5, how["norm"], how["dh"] if train else None, how["dy"] if train else None)
    args = dict(post_scale=c["post"], post_bias=c["post_bias"], pre_scale=c["pre"], pre_bias=c["pre_bias"],
                gate=c["gate"], residual_scale=c["alpha"], norm=c["norm"])
    h, y, stats = gs.residual_norm(X, F, return_stats=True, **args)
    close(h, *want["h"], "h")
    close(stats, *want["stats"], "stats")
    assert (y is None) == (c["pre"] is None)
    if y is not None:
        close(y, *want["y"], "y")
    plain = gs.residual_norm(X, F, **args)
    assert torch.equal(plain[0], h) and (y is None or torch.equal(plain[1], y))
    if not train:
        return
    names = ("dx", "dbranch", "dgate", "dpost", "dpost_bias", "dpre", "dpre_bias")
    got = gs.residual_norm_backward(c["dh"], c["dy"], X, F, stats, **args)
    layer = c["norm"] == "layer"
    there = dict(dx=True, dbranch=True, dgate=c["gate"] is not None, dpost=c["post"] is not None,
                 dpost_bias=c["post"] is not None and (layer or c["post_bias"] is not None), dpre=c["pre"] is not None,
                 dpre_bias=c["pre"] is not None and (layer or c["pre_bias"] is not None))
    for name, v in zip(names, got):
        assert (v is not None) == there[name], name
        if v is not None:
            close(v, *want[name], name)
    again = gs.residual_norm_backward(c["dh"], c["dy"], X, F, stats, **args)
    assert all(p is None or torch.equal(p, q) for p, q in zip(got, again))


def join_inputs(r, shape, t, pt, norm, post=True, pre=True, bias=True, gate="none", alpha=1.0, dh=True):
    n = shape[-1]
    lead = {"none": None, "channel": (), "sequence": shape[:1], "token": shape[:-1]}[gate]
    return r(*shape, mean=0.3, t=t), r(*shape, scale=0.7, mean=-0.2, t=t), {
        "post": r(n, scale=0.3, mean=1.0, t=pt) if post else None, "post_bias": r(n, t=pt) if post and bias else None,
        "pre": r(n, scale=0.3, mean=1.0, t=pt) if pre else None, "pre_bias": r(n, t=pt) if pre and bias else None,
        "gate": None if lead is None else r(*lead, n, scale=0.5, mean=0.5, t=pt), "alpha": alpha, "norm": norm,
        "dh": r(*shape, t=t) if dh else None, "dy": r(*shape, t=t) if pre else None}


JOINS = [(1, 1, 8), (2, 3, 7), (1, 5, 64), (3, 2, 65), (2, 40, 256), (1, 9, 257), (3, 7, 512), (2, 5, 777),
         (1, 4, 1024), (4, 33, 1032), (2, 3, 2048), (1, 3, 2049), (1, 2, 4096), (1, 3, 5000), (1, 2, 8192),
         (1, 2, 9000), (1, 1, 16384), (600, 3, 24), (1, 1500, 40), (3, 1, 16383)]


@pytest.mark.parametrize("shape", JOINS)
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("dtype,params", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32")])
def test_residual_norm(gs, shape, norm, dtype, params):
    r = maker(sum(shape))
    gate = ["none", "channel", "sequence", "token"][sum(shape) % 4]
    check_join(gs, *join_inputs(r, shape, TYPES[dtype], TYPES[params], norm, gate=gate, alpha=0.75))


@pytest.mark.parametrize("gate", ["none", "channel", "sequence", "token"])
@pytest.mark.parametrize("post,pre,bias,dh", [(True, True, False, True), (True, False, True, True),
                                              (False, True, True, False), (False, False, False, True)])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_residual_norm_of_every_part(gs, gate, post, pre, bias, dh, norm):
    for dtype, params, shape in (("f32", "f32", (3, 37, 72)), ("bf16", "bf16", (2, 300, 264)),
                                 ("f16", "f32", (700, 2, 40))):
        r = maker(11)
        check_join(gs, *join_inputs(r, shape, TYPES[dtype], TYPES[params], norm, post, pre, bias, gate, 1.5, dh))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_residual_norm_strides_alignment_and_shapes(gs, dtype):
    t, r = TYPES[dtype], maker(6)
    wide, other = r(4, 6, 200, t=t), r(4, 6, 200, t=t)
    for lo in (0, 3, 8):
        x, f = wide[..., lo:lo + 96], other[:, :1, lo:lo + 96].expand(4, 6, 96)
        _, _, how = join_inputs(r, (4, 6, 96), t, torch.float32, "layer", gate="sequence")
        check_join(gs, x, f, how, gpu=(wide.cuda()[..., lo:lo + 96], other.cuda()[:, :1, lo:lo + 96].expand(4, 6, 96)))
    x, f, how = join_inputs(r, (96,), t, torch.float32, "rms", gate="channel")
    check_join(gs, x, f, how)


def test_residual_norm_of_constant_rows_and_nan(gs):
    """A constant row has no deviation; a NaN or an infinity stays in its row."""
    cols = 1177
    x, f = torch.full((4, cols), 1e4, device="cuda"), torch.zeros(4, cols, device="cuda")
    w, b = torch.ones(cols, device="cuda"), torch.arange(float(cols), device="cuda")
    h, y = gs.residual_norm(x, f, pre_scale=w, pre_bias=b, norm="layer")
    assert torch.equal(y, b.expand(4, cols)) and torch.equal(h, x)
    x = torch.randn(4, cols, device="cuda")
    h, y, stats = gs.residual_norm(x, f, pre_scale=w, post_scale=w, return_stats=True)
    x2 = x.clone()
    x2[1, 3], x2[2, 4] = math.nan, math.inf
    h2, y2, stats2 = gs.residual_norm(x2, f, pre_scale=w, post_scale=w, return_stats=True)
    assert y2[1].isnan().all() and y2[2, 4].isnan() and torch.equal(y2[0], y[0]) and torch.equal(y2[3], y[3])
    d = torch.randn(4, cols, device="cuda")
    got = gs.residual_norm_backward(d, d, x2, f, stats2, pre_scale=w, post_scale=w)
    want = gs.residual_norm_backward(d, d, x, f, stats, pre_scale=w, post_scale=w)
    for p, q in zip(got[:2], want[:2]):
        assert torch.equal(p[0], q[0]) and torch.equal(p[3], q[3])


def test_residual_norm_without_rows(gs):
    x, w = torch.empty(0, 5, 16, device="cuda"), torch.ones(16, device="cuda")
    h, y, stats = gs.residual_norm(x, x, pre_scale=w, post_scale=w, gate=w, return_stats=True)
    used = [torch.full((16,), 7.0, device="cuda") for _ in range(4)]
    del used
    dx, df, dgate, dpost, _, dpre, _ = gs.residual_norm_backward(h, y, x, x, stats, pre_scale=w, post_scale=w, gate=w)
    assert dx.shape == x.shape and not dgate.any() and not dpost.any() and not dpre.any()


# ------------------------------------------------------- gated recurrence

def check_recurrence(gs, x, g, state=None, lengths=None, dy=None, dlast=None, gpu=None):
    want = ref.recurrence(x, g, state, lengths, dy, dlast)
    X, G, dY = gpu or (x.cuda(), g.cuda(), None if dy is None else dy.cuda())
    S, N, dS = (None if v is None else v.cuda() for v in (state, lengths, dlast))
    y, last, saved = gs.gated_recurrence(X, G, S, N, return_saved=True)
    close(y, *want["y"], "y")
    close(last, *want["last"], "last")
    plain = gs.gated_recurrence(X, G, S, N)
    assert torch.equal(plain[0], y) and torch.equal(plain[1], last)
    if S is not None:
        kept = S.clone()                             # a state kept from call to call
        y2, last2 = gs.gated_recurrence(X, G, kept, N, last=kept)
        assert last2 is kept and torch.equal(kept, last) and torch.equal(y2, y)
    if dy is None:
        return
    got = gs.gated_recurrence_backward(dY, X, G, saved, dS, N)
    for name, v in zip(("dx", "dg", "dstate"), got):
        close(v, *want[name], name)
    again = gs.gated_recurrence_backward(dY, X, G, saved, dS, N)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


SCANS = [(1, 1, 1), (2, 1, 64), (3, 2, 5), (1, 15, 130), (2, 16, 128), (2, 17, 2), (1, 127, 66), (2, 128, 64),
         (1, 129, 200), (3, 255, 33), (2, 256, 8), (1, 700, 70), (2, 1500, 3), (1, 5000, 65), (17, 40, 24),
         (300, 3, 8)]


@pytest.mark.parametrize("shape", SCANS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("mean", [0.0, 4.0])
def test_gated_recurrence(gs, shape, dtype, mean):
    t, r = TYPES[dtype], maker(sum(shape))
    B, _, C = shape
    check_recurrence(gs, r(*shape, t=t), r(*shape, scale=1.5, mean=mean, t=t), r(B, C), None, r(*shape, t=t), r(B, C))


@pytest.mark.parametrize("shape", [(5, 1, 6), (5, 40, 130), (5, 300, 33), (5, 1400, 64)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gated_recurrence_lengths(gs, shape, dtype):
    """Sequences of no, one and more tokens; what lies past a length is NaN, and held lengths past the ends."""
    t, r = TYPES[dtype], maker(9)
    B, L, C = shape
    n = torch.tensor([0, 1, L, max(1, L // 2), -3], dtype=torch.int32)
    x, g, dy = r(*shape, t=t), r(*shape, scale=1.5, mean=1.0, t=t), r(*shape, t=t)
    past = (torch.arange(L) >= n.clamp(0, L)[:, None])[..., None]
    x, g, dy = (torch.where(past, torch.tensor(math.nan, dtype=t), v) for v in (x, g, dy))
    check_recurrence(gs, x, g, r(B, C), n, dy, r(B, C))
    n[2] = L + 7
    check_recurrence(gs, x, g, None, n, dy, None)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_gated_recurrence_strides_and_alignment(gs, dtype):
    """Channels off their alignment, gaps, tokens first, a broadcast sequence."""
    t, r = TYPES[dtype], maker(12)
    wide = [r(3, 150, 90, t=t) for _ in range(3)]
    for lo in (0, 1, 2):
        cpu = [v[..., lo:lo + 66] for v in wide]
        check_recurrence(gs, *cpu[:2], None, None, cpu[2], None, gpu=[v.cuda()[..., lo:lo + 66] for v in wide])
    first = [v.transpose(0, 1) for v in wide]
    check_recurrence(gs, *first[:2], None, None, first[2], None,
                     gpu=[v.cuda().transpose(0, 1) for v in wide])
    one = [v[:1].expand(3, 150, 90) for v in wide]
    check_recurrence(gs, *one[:2], None, None, one[2], None, gpu=[v.cuda()[:1].expand(3, 150, 90) for v in wide])


def test_gated_recurrence_of_extreme_gates(gs):
    """Gates that are 0 or 1 in fp32, infinities among them: a state that is kept, or replaced."""
    x = torch.arange(1.0, 13.0, device="cuda").reshape(1, 12, 1)
    g = torch.tensor([200.0, -200.0, math.inf, -math.inf, 88.0, -88.0, 104.0, -104.0, 1e30, -1e30, 0.0, 50.0])
    state = torch.tensor([[5.0]], device="cuda")
    y, last, saved = gs.gated_recurrence(x, g.cuda().reshape(1, 12, 1), state, return_saved=True)
    assert y.flatten().tolist()[:10] == [5, 2, 2, 4, 4, 6, 6, 8, 8, 10]
    assert y.flatten().tolist()[10:] == [10.5, 10.5] and last.item() == 10.5
    dx, dg, dstate = gs.gated_recurrence_backward(torch.ones_like(x), x, g.cuda().reshape(1, 12, 1), saved)
    assert dx.isfinite().all() and dg.isfinite().all() and dstate.item() == 1.0


def test_gated_recurrence_nan_stays_in_its_channel(gs):
    r = maker(2)
    x, g = r(2, 700, 70).cuda(), r(2, 700, 70).cuda()
    y, last = gs.gated_recurrence(x, g)
    x[1, 300, 5] = math.nan
    got, got_last = gs.gated_recurrence(x, g)
    assert got[1, 300:, 5].isnan().all() and got_last[1, 5].isnan()
    got[1, 300:, 5], got_last[1, 5] = y[1, 300:, 5], last[1, 5]
    assert torch.equal(got, y) and torch.equal(got_last, last)


def test_gated_recurrence_without_tokens(gs):
    x, state = torch.empty(2, 0, 6, device="cuda"), torch.randn(2, 6, device="cuda")
    y, last, saved = gs.gated_recurrence(x, x, state, return_saved=True)
    assert y.shape == x.shape and torch.equal(last, state)
    dx, dg, dstate = gs.gated_recurrence_backward(x, x, x, saved, state)
    assert torch.equal(dstate, state) and dx.shape == x.shape
    assert gs.gated_recurrence(torch.empty(0, 5, 6, device="cuda"), torch.empty(0, 5, 6, device="cuda"))[1].shape == (
        0, 6)


def test_gated_recurrence_step_by_step_is_the_whole_sequence(gs):
    """One token at a time, the state kept in place, against one call: the same values up to fp32's roundings."""
    r = maker(5)
    x, g = r(3, 70, 130).cuda(), r(3, 70, 130, mean=1.0).cuda()
    want = ref.recurrence(x.cpu(), g.cpu())
    state = torch.zeros(3, 130, device="cuda")
    steps = [gs.gated_recurrence(x[:, i:i + 1], g[:, i:i + 1], state, last=state)[0] for i in range(70)]
    close(torch.cat(steps, 1), *want["y"], "y")
    close(state, *want["last"], "last")
