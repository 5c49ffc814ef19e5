"""The block operators on the GPU where a layout, a stream or a size is out of the ordinary: streams given by name,
captured graphs, workspaces, long sequences in parts, tensors past 2^31 elements.  Bounds are block_reference's."""

import ctypes
import math

import pytest
import torch

import block_reference as ref
from test_gpu_blocks import check_gated, check_recurrence, join_inputs, maker
from test_gpu_tokens import TYPES, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import spatial_transformer_grid_amd as gs

    gs.token_lib()
    return gs


# ------------------------------------------------------- streams and graphs

def every_call(gs, t, stream=None):
    """A function that makes every call once on the same inputs and returns all outputs."""
    r = maker(31)
    x, w, u, dy = (r(90, 72, t=t), r(100, 72, scale=0.12, t=t), r(100, 72, scale=0.12, t=t), r(90, 100, t=t))
    xo, wo, uo, dyo = (v.cuda() for v in (r(90, 75, t=t), r(61, 75, scale=0.1, t=t), r(61, 75, scale=0.1, t=t), r(90, 61, t=t)))
    x, w, u, dy = (v.cuda() for v in (x, w, u, dy))
    jx, jf, how = join_inputs(r, (3, 50, 96), t, torch.float32, "layer", gate="sequence", alpha=0.5)
    jx, jf = jx.cuda(), jf.cuda()
    how = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in how.items()}
    args = dict(post_scale=how["post"], post_bias=how["post_bias"], pre_scale=how["pre"], pre_bias=how["pre_bias"],
                gate=how["gate"], residual_scale=how["alpha"], norm="layer")
    sx, sg, sdy = (r(2, 5000, 24, t=t).cuda() for _ in range(3))
    state, dlast = r(2, 24).cuda(), r(2, 24).cuda()
    n = torch.tensor([5000, 3100], dtype=torch.int32, device="cuda")
    k = {} if stream is None else {"stream": stream}

    def calls():
        out = []
        for a, b, c, d in ((x, w, u, dy), (x[:9], w, u, dy[:9]), (xo, wo, uo, dyo)):
            y, saved = gs.gated_linear(a, b, c, "gelu", return_saved=True, **k)
            out += [y, saved, *gs.gated_linear_backward(d, a, b, c, saved, "gelu", **k)]
        h, y, stats = gs.residual_norm(jx, jf, return_stats=True, **args, **k)
        out += [h, y, stats, *gs.residual_norm_backward(how["dh"], how["dy"], jx, jf, stats, **args, **k)]
        for a, b, d, lengths in ((sx, sg, sdy, n), (sx[:, :70], sg[:, :70], sdy[:, :70], None)):
            y, last, saved = gs.gated_recurrence(a, b, state, lengths, return_saved=True, **k)
            # (the states of chunks that a sequence does not reach are not written)
            out += [y, last, *gs.gated_recurrence_backward(d, a, b, saved, dlast, lengths, **k)]
        return out
    return calls


@pytest.mark.parametrize("dtype", list(TYPES))
def test_calls_on_a_stream_given_by_name(gs, dtype):
    """Inputs that the current stream is still writing, and a busy named stream: the bits of plain calls."""
    t = TYPES[dtype]
    want = every_call(gs, t)()
    square = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(5):
            torch.mm(square, square)
    got = every_call(gs, t, s)()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_in_a_captured_graph(gs, dtype):
    """Every replay equals the eager calls, with eager calls and other work between the replays."""
    calls = every_call(gs, TYPES[dtype])
    want = calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for i in range(4):
        for v in held:
            if v.is_floating_point():
                v.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), i
        assert all(torch.equal(a, b) for a, b in zip(want, calls()))


def test_graphs_that_share_a_workspace(gs):
    """Two captured graphs that name one scratch tensor, replayed in turn on one stream."""
    r = maker(4)
    scratch = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN, whatever type reads it
    x, w, u, dy = (v.cuda() for v in (r(80, 70), r(50, 70, scale=0.1), r(50, 70, scale=0.1), r(80, 50)))
    sx, sg, sdy = (r(1, 6000, 40).cuda() for _ in range(3))

    def gated():
        y, saved = gs.gated_linear(x, w, u, return_saved=True, workspace=scratch)
        return [y, *gs.gated_linear_backward(dy, x, w, u, saved, workspace=scratch)]

    def scan():
        y, last, saved = gs.gated_recurrence(sx, sg, return_saved=True, workspace=scratch)
        return [y, last, *gs.gated_recurrence_backward(sdy, sx, sg, saved, workspace=scratch)]
    want, graphs = [gated(), scan()], []
    for f in (gated, scan):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = f()
        graphs.append((g, held))
    for _ in range(3):
        scratch.fill_(0xFF)
        for (g, held), v in zip(graphs, want):
            g.replay()
        torch.cuda.synchronize()
        for (g, held), v in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(held, v))


# --------------------------------------------------------------- workspaces

@pytest.mark.parametrize("dtype", list(TYPES))
def test_without_a_workspace(gs, dtype):
    """The forward calls run without scratch memory, and with too little."""
    t, r = TYPES[dtype], maker(9)
    for rows, width, hidden in ((70, 1500, 40), (130, 75, 33), (100, 2048, 64)):
        x, w, u = r(rows, width, t=t), r(hidden, width, scale=width ** -0.5, t=t), r(hidden, width, scale=width ** -0.5, t=t)
        want = ref.gated(x, w, u, "silu")
        for scratch in (torch.empty(0, dtype=torch.uint8, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")):
            close(gs.gated_linear(x.cuda(), w.cuda(), u.cuda(), workspace=scratch), *want["y"], "y")
    x, g, dy = (r(1, 4000, 20, t=t) for _ in range(3))
    want = ref.recurrence(x, g, None, None, dy)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    y, last, saved = gs.gated_recurrence(x.cuda(), g.cuda(), return_saved=True, workspace=none)
    close(y, *want["y"], "y")
    got = gs.gated_recurrence_backward(dy.cuda(), x.cuda(), g.cuda(), saved, workspace=none)
    for name, v in zip(("dx", "dg", "dstate"), got):
        close(v, *want[name], name)


def test_small_workspaces_are_refused(gs):
    r = maker(1)
    x, w, dy = r(70, 32).cuda(), r(40, 32).cuda(), r(70, 40).cuda()
    y, saved = gs.gated_linear(x, w, w, return_saved=True)
    small = torch.empty(512, dtype=torch.uint8, device="cuda")
    with pytest.raises(gs.GSError):
        gs.gated_linear_backward(dy, x, w, w, saved, workspace=small)
    s = torch.ones(32, device="cuda")
    h, y, stats = gs.residual_norm(x, x, s, s, return_stats=True)
    with pytest.raises(gs.GSError):
        gs.residual_norm_backward(x, x, x, x, stats, s, s, workspace=small[:256])
    with pytest.raises(ValueError):
        gs.residual_norm_backward(x, x, x, x, stats, s, s, workspace=torch.empty(1 << 20, dtype=torch.uint8))


# -------------------------------------------------------------- gated sizes

@pytest.mark.parametrize("rows,width,hidden", [(66, 64, 40), (129, 65, 128), (255, 128, 63), (300, 40, 700), (65, 1030, 72),
                                               (1030, 72, 65), (640, 640, 640), (2049, 24, 2056), (70, 16, 5000)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gated_linear_of_every_tile(gs, rows, width, hidden, dtype):
    """Tiles of 64, 128 and 256, cut sums, edges of all of them, chunks that end inside a row."""
    t, r = TYPES[dtype], maker(rows + hidden)
    check_gated(gs, r(rows, width, t=t), r(hidden, width, scale=width ** -0.5, t=t),
                r(hidden, width, scale=width ** -0.5, t=t), "silu", r(rows, hidden, t=t))


@pytest.mark.parametrize("rows", [3, 40, 1300])
def test_gated_linear_operands_off_their_alignment(gs, rows):
    """16-bit rows that begin at odd elements, with a width of whole chunks: the kernel for few rows takes them."""
    t, r = torch.bfloat16, maker(2)
    big = r(rows, 100, t=t).cuda()
    w = r(2 * 64 * 96 + 1, scale=0.1, t=t).cuda()
    x, wg, wu = big[:, 1:97], w[1:1 + 64 * 96].view(64, 96), w[1 + 64 * 96:].view(64, 96)
    check_gated(gs, x.cpu(), wg.cpu(), wu.cpu(), "silu", r(rows, 64, t=t), X=x)
    y, saved = gs.gated_linear(x, wg, wu, return_saved=True)
    want = ref.gated(x.cpu(), wg.cpu(), wu.cpu(), "silu")
    close(y, *want["y"], "y")


def test_gated_linear_gradients_apart(gs):
    """dX alone and the weights' gradients alone are those of the whole call, by the C entry."""
    r, lib = maker(12), gs.token_lib()
    for t, code in ((torch.float32, 0), (torch.bfloat16, 2)):
        x, w, u, dy = (v.cuda() for v in (r(70, 40, t=t), r(90, 40, t=t), r(90, 40, t=t), r(70, 90, t=t)))
        _, saved = gs.gated_linear(x, w, u, return_saved=True)
        want = gs.gated_linear_backward(dy, x, w, u, saved)
        need = ctypes.c_int64(0)
        assert lib.gs_gated_linear_backward_workspace_size(code, 70, 40, 90, ctypes.byref(need)) == 0
        ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        for input_too, weights_too in ((True, False), (False, True)):
            ws.fill_(0xFF)
            dx, dg, du = torch.full_like(x, 7), torch.full_like(w, 7), torch.full_like(u, 7)
            st = lib.gs_gated_linear_backward(
                dy.data_ptr(), x.data_ptr(), code, 70, 40, 90, 90, 40, w.data_ptr(), u.data_ptr(), 0, saved.data_ptr(),
                dx.data_ptr() if input_too else None, 40, dg.data_ptr() if weights_too else None,
                du.data_ptr() if weights_too else None, ws.data_ptr(), need.value, stream)
            assert st == 0
            assert torch.equal(dx, want[0] if input_too else torch.full_like(x, 7))
            assert torch.equal(dg, want[1] if weights_too else torch.full_like(w, 7))
            assert torch.equal(du, want[2] if weights_too else torch.full_like(u, 7))


# ---------------------------------------------------- sequences in parts

@pytest.mark.parametrize("shape", [(1, 2049, 1), (1, 2200, 130), (2, 4500, 33), (3, 6000, 8), (1, 9000, 16), (5, 2500, 70)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gated_recurrence_in_parts(gs, shape, dtype):
    """Long sequences of few channels, with states at both ends, lengths inside a part, at its border and none."""
    t, r = TYPES[dtype], maker(sum(shape))
    B, L, C = shape
    x, g, dy = r(*shape, t=t), r(*shape, scale=1.5, mean=2.0, t=t), r(*shape, t=t)
    check_recurrence(gs, x, g, r(B, C), None, dy, r(B, C))
    n = torch.tensor(([L // 3, 1024, L, 0, 1] * B)[:B], dtype=torch.int32)
    past = (torch.arange(L) >= n[:, None])[..., None]
    x, g, dy = (torch.where(past, torch.tensor(math.nan, dtype=t), v) for v in (x, g, dy))
    check_recurrence(gs, x, g, r(B, C), n, dy, r(B, C))


def test_gated_recurrence_states_in_place_in_both_directions(gs):
    """last over state, and dstate over dlast, where the tokens are split over blocks."""
    r, lib = maker(7), gs.token_lib()
    x, g, dy = (r(1, 8192, 24).cuda() for _ in range(3))
    state, dlast = r(1, 24).cuda(), r(1, 24).cuda()
    y, last, saved = gs.gated_recurrence(x, g, state, return_saved=True)
    kept = state.clone()
    assert torch.equal(gs.gated_recurrence(x, g, kept, last=kept)[0], y) and torch.equal(kept, last)
    dx, dg, dstate = gs.gated_recurrence_backward(dy, x, g, saved, dlast)
    d = gs.blocks.RecurrenceDesc(0, 1, 8192, 24, *[(8192 * 24, 24)] * 6)
    need = ctypes.c_int64(0)
    assert lib.gs_gated_recurrence_backward_workspace_size(ctypes.byref(d), ctypes.byref(need)) == 0 and need.value > 0
    ws, ox, og, kept = torch.empty(need.value, dtype=torch.uint8, device="cuda"), torch.empty_like(x), torch.empty_like(
        x), dlast.clone()
    assert lib.gs_gated_recurrence_backward(ctypes.byref(d), dy.data_ptr(), x.data_ptr(), g.data_ptr(), saved.data_ptr(),
                                            kept.data_ptr(), None, ox.data_ptr(), og.data_ptr(), kept.data_ptr(),
                                            ws.data_ptr(), need.value, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(ox, dx) and torch.equal(og, dg) and torch.equal(kept, dstate)


def test_gated_recurrence_from_one_call_to_the_next(gs):
    """A sequence in three calls that hand the state on, and its gradients in three calls back."""
    r = maker(8)
    x, g, dy = (r(2, 700, 40).cuda() for _ in range(3))
    want = ref.recurrence(x.cpu(), g.cpu(), None, None, dy.cpu())
    cuts, state, saved, ys = ((0, 100), (100, 350), (350, 700)), None, [], []
    for a, b in cuts:
        y, state, s = gs.gated_recurrence(x[:, a:b], g[:, a:b], state, return_saved=True)
        ys.append(y)
        saved.append(s)
    close(torch.cat(ys, 1), *want["y"], "y")
    d, dxs, dgs = None, [], []
    for (a, b), s in zip(cuts[::-1], saved[::-1]):
        dx, dg, d = gs.gated_recurrence_backward(dy[:, a:b], x[:, a:b], g[:, a:b], s, d)
        dxs.insert(0, dx)
        dgs.insert(0, dg)
    close(torch.cat(dxs, 1), *want["dx"], "dx")
    close(torch.cat(dgs, 1), *want["dg"], "dg")
    close(d, *want["dstate"], "dstate")


# ----------------------------------------------- tensors past 2^31 elements

def test_gated_recurrence_past_2_to_the_31(gs):
    B, L, C = 3, 1 << 19, 1400
    x = torch.empty(B, L, C, dtype=torch.bfloat16, device="cuda")
    g = torch.empty_like(x)
    for b in range(B):
        x[b].normal_()
        g[b].normal_(1.0)
    y, last, saved = gs.gated_recurrence(x, g, return_saved=True)
    # the last tokens of the last sequence from a state some way before them, which a product of gates near 0.7 forgets
    at = L - 200
    for sl in (slice(0, 40), slice(C - 40, C)):
        want = ref.recurrence(x[2:, at:, sl].cpu(), g[2:, at:, sl].cpu(), saved[2:, at // 64, sl].cpu() if at % 64 == 0 else None)
        first = 150                                  # 150 gates' product is below 1e-12
        close(y[2:, at + first:, sl], *(v[:, first:] for v in want["y"]), "y")
    dx, dg, dstate = gs.gated_recurrence_backward(y, x, g, saved)
    for sl in (slice(0, 40), slice(C - 40, C)):
        want = ref.recurrence(x[2:, at:, sl].cpu(), g[2:, at:, sl].cpu(), None, None, y[2:, at:, sl].cpu())
        close(dx[2:, at + 150:, sl], *(v[:, 150:] for v in want["dx"]), "dx")


def test_residual_norm_past_2_to_the_31(gs):
    rows, cols = (1 << 18) + 9, 8200
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(cols, device="cuda")
    h, y, stats = gs.residual_norm(x, x, w, w, gate=w, return_stats=True)
    ends = torch.tensor([0, 1, rows - 2, rows - 1], device="cuda")
    want = ref.join(x[ends].cpu()[None], x[ends].cpu()[None], w.cpu(), None, w.cpu(), None, w.cpu(), 1.0, 1e-5, "rms",
                    x[ends].cpu()[None], y[ends].cpu()[None])
    close(h[ends][None], *want["h"], "h")
    close(y[ends][None], *want["y"], "y")
    dx, df, *_ = gs.residual_norm_backward(x, y, x, x, stats, w, w, gate=w)
    close(dx[ends][None], *want["dx"], "dx")
    close(df[ends][None], *want["dbranch"], "dbranch")


def test_gated_linear_past_2_to_the_31(gs):
    rows, width, hidden = 1 << 17, 16, (1 << 14) + 24
    r, t = maker(3), torch.bfloat16
    x = torch.empty(rows, width, dtype=t, device="cuda").normal_()
    w, u = r(hidden, width, scale=0.25, t=t).cuda(), r(hidden, width, scale=0.25, t=t).cuda()
    y, saved = gs.gated_linear(x, w, u, return_saved=True)
    ends = torch.tensor([0, 1, rows - 2, rows - 1], device="cuda")
    want = ref.gated(x[ends].cpu(), w.cpu(), u.cpu(), "silu", y[ends].cpu())
    close(y[ends], *want["y"], "y")
    close(saved[1][ends], *want["b"], "b")
    dx, dg, du = gs.gated_linear_backward(y, x, w, u, saved)
    close(dx[ends], *want["dx"], "dx")
    assert dg.isfinite().all() and du.isfinite().all()


def test_gated_linear_rows_further_apart_than_a_tiles_offsets(gs):
    """Rows of a wide buffer, more than 4 MiB apart, give the bits of the same rows side by side."""
    apart = (1 << 21) + 8
    x = torch.randn(66, 64, device="cuda").to(torch.bfloat16)
    wide = torch.zeros(66 * apart, dtype=torch.bfloat16, device="cuda").as_strided((66, 64), (apart, 1))
    wide.copy_(x)
    wg, wu = (torch.randn(48, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    y, saved = gs.gated_linear(x, wg, wu, return_saved=True)
    z, again = gs.gated_linear(wide, wg, wu, return_saved=True)
    assert torch.equal(z, y) and torch.equal(again, saved)
    for p, q in zip(gs.gated_linear_backward(y, wide, wg, wu, saved), gs.gated_linear_backward(y, x, wg, wu, saved)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 66])
def test_gated_linear_gradients_of_infinities(gs, rows, dtype):
    """With positive operands an infinite dY gives infinite gradients, no NaN, also where what the rounding of da and
    db left is multiplied too; so does one whose da passes the element type's range."""
    t = TYPES[dtype]
    x, w = torch.ones(rows, 16, device="cuda", dtype=t), torch.full((24, 16), 0.25, device="cuda", dtype=t)
    y, saved = gs.gated_linear(x, w, w, return_saved=True)
    for value in (math.inf, 0.9 * torch.finfo(t).max):
        dy = torch.zeros(rows, 24, device="cuda", dtype=t)
        dy[0] = value
        for v in gs.gated_linear_backward(dy, x, w, w, saved):
            assert torch.isposinf(v[0]).all() and not torch.isnan(v).any()
