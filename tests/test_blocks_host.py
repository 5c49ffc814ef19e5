"""The operators around a block without a GPU: the 64-bit reference against torch's
gradients and differences, the descriptors' layout, and refusals (every call here
fails validation or has nothing to do)."""

import ctypes
import math
import os
import subprocess

import pytest
import torch

import block_reference as ref
from conftest import ROOT

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails before


@pytest.fixture(scope="module")
def tk():
    from spatial_transformer_grid_amd import _binding, _tokens

    if not os.path.exists(_binding.LIB_PATH):
        from spatial_transformer_grid_amd import build

        build.build()
    return _tokens


# ------------------------------------------------------------- reference

def leaves(seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g, dtype=torch.float64, requires_grad=True) for s in shapes]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_reference_gated_is_torchs(act):
    x, wg, wu, dy = leaves(1, (5, 4), (6, 4), (6, 4), (5, 6))
    fn = torch.nn.functional
    f = {"silu": fn.silu, "gelu": fn.gelu, "gelu_tanh": lambda v: fn.gelu(v, approximate="tanh"), "relu": fn.relu}[act]
    y = f(x @ wg.t()) * (x @ wu.t())
    grads = torch.autograd.grad(y, (x, wg, wu), dy)
    got = ref.gated(x.detach(), wg.detach(), wu.detach(), act, dy.detach())
    for name, v in zip(("y", "dx", "dgate", "dup"), (y, *grads)):
        assert torch.allclose(got[name][0], v, atol=1e-12), name


@pytest.mark.parametrize("gate", [None, (7,), (2, 7), (2, 3, 7)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_reference_join_is_torchs(gate, kind, post, pre):
    x, f, w1, b1, w2, b2, m, dh, dy = leaves(2, (2, 3, 7), (2, 3, 7), 7, 7, 7, 7, gate or (1,), (2, 3, 7), (2, 3, 7))

    def norm(z, w, b):
        z = z - z.mean(-1, keepdim=True) if kind == "layer" else z
        return z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * w + b
    eps = float(torch.tensor(1e-5, dtype=torch.float32))
    p = norm(f, w1, b1) if post else f
    p = p if gate is None else p * (m.unsqueeze(1) if m.dim() == 2 else m)
    h = 1.25 * x + p
    out, back = [h], [dh]
    if pre:
        out.append(norm(h, w2, b2))
        back.append(dy)
    at = {"dx": x, "dbranch": f, "dgate": m, "dpost": w1, "dpost_bias": b1, "dpre": w2, "dpre_bias": b2}
    there = [n for n in at if not (n == "dgate" and gate is None) and not ("post" in n and not post) and not (
        "pre" in n and not pre)]
    grads = torch.autograd.grad(out, [at[n] for n in there], back)
    d = [v.detach() for v in (x, f, w1, b1, w2, b2, m, dh, dy)]
    got = ref.join(d[0], d[1], *(d[2:4] if post else (None, None)), *(d[4:6] if pre else (None, None)),
                   None if gate is None else d[6], 1.25, 1e-5, kind, d[7], d[8] if pre else None)
    assert torch.allclose(got["h"][0], h)
    for n, v in zip(there, grads):
        assert torch.allclose(got[n][0], v, atol=1e-10), n


def test_reference_recurrence_against_differences():
    x, g, state, dy, dlast = (v.detach() for v in leaves(3, (2, 5, 3), (2, 5, 3), (2, 3), (2, 5, 3), (2, 3)))
    n = torch.tensor([5, 3], dtype=torch.int32)
    got = ref.recurrence(x, g, state, n, dy, dlast)
    hold = (torch.arange(5) < n[:, None])[..., None]
    assert (got["y"][0][~hold.expand(2, 5, 3)] == 0).all()
    at = {"dx": x, "dg": g, "dstate": state}
    for name, t in at.items():
        for i in range(t.numel()):
            vals = []
            for sign in (1, -1):
                moved = {k: v.clone() for k, v in at.items()}
                moved[name].view(-1)[i] += sign * 1e-5
                r = ref.recurrence(moved["dx"], moved["dg"], moved["dstate"], n)
                vals.append((r["y"][0] * dy).sum() + (r["last"][0] * dlast).sum())
            # h^2 times third derivatives of order one, rounding 1e-16 / h
            assert abs((vals[0] - vals[1]) / 2e-5 - got[name][0].view(-1)[i]) < 1e-8, (name, i)


# ------------------------------------------------------------------- ABI

@pytest.mark.parametrize("name,struct", [("gs_residual_norm_desc", "ResidualNormDesc"),
                                         ("gs_recurrence_desc", "RecurrenceDesc")])
def test_descriptor_layout(tk, tmp_path, name, struct):
    from spatial_transformer_grid_amd import blocks

    cls = getattr(blocks, struct)
    fields = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gsample_tokens.h"\nint main(void) {\n' +
                   "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (name, f) for f in fields) +
                   'printf("%%zu\\n%%d\\n", sizeof(%s), GS_RECURRENCE_CHUNK); return 0; }\n' % name)
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe],
                   check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f in fields] + [ctypes.sizeof(cls), blocks.RECURRENCE_CHUNK]


def size_of(call, *args):
    need = ctypes.c_int64(-1)
    status = call(*args, ctypes.byref(need))
    return need.value if status == 0 else -status


def test_gated_linear_refuses(tk):
    lib = tk.token_lib()

    def fwd(x=FAKE, dtype=0, rows=4, width=8, hidden=16, xs=8, wg=FAKE, wu=FAKE, act=0, y=FAKE, ys=16, ws=None, n=0):
        return lib.gs_gated_linear(x, dtype, rows, width, hidden, xs, wg, wu, act, y, ys, None, ws, n, None)

    bad = [(dict(x=None), 1), (dict(wg=None), 1), (dict(wu=None), 1), (dict(y=None), 1), (dict(rows=-1), 2),
           (dict(width=-1), 2), (dict(hidden=-1), 2), (dict(width=0), 2), (dict(xs=-1), 2), (dict(ys=15), 2),
           (dict(dtype=3), 3), (dict(dtype=-1), 3), (dict(act=4), 4), (dict(act=-1), 4), (dict(n=-1), 4),
           (dict(ws=ctypes.c_void_p(0x1010), n=512), 4), (dict(rows=2 ** 20 + 1), 6), (dict(width=2 ** 20 + 1), 6),
           (dict(hidden=2 ** 20 + 1, ys=2 ** 23), 6), (dict(rows=2 ** 20, hidden=2 ** 17, ys=2 ** 17), 6),
           (dict(hidden=2 ** 20, width=2 ** 20, rows=2 ** 16, ys=2 ** 20), 6)]
    for kw, status in bad:
        assert fwd(**kw) == status, kw
    assert fwd(rows=0, x=None, y=None) == 0 and fwd(hidden=0, wg=None, wu=None, y=None) == 0
    assert lib.gs_gated_linear_workspace_size(0, 4, 8, 16, None) == 1
    assert size_of(lib.gs_gated_linear_workspace_size, 0, -1, 8, 16) == -2
    assert size_of(lib.gs_gated_linear_workspace_size, 5, 4, 8, 16) == -3
    need = size_of(lib.gs_gated_linear_backward_workspace_size, 0, 4, 8, 16)
    assert need > 0

    def bwd(dy=FAKE, x=FAKE, rows=4, width=8, hidden=16, dys=16, xs=8, wg=FAKE, wu=FAKE, act=0, saved=FAKE, dx=FAKE,
            dxs=8, dwg=FAKE, dwu=FAKE, ws=FAKE, n=need):
        return lib.gs_gated_linear_backward(dy, x, 0, rows, width, hidden, dys, xs, wg, wu, act, saved, dx, dxs, dwg, dwu,
                                            ws, n, None)

    for kw, status in [(dict(dy=None), 1), (dict(x=None), 1), (dict(wg=None), 1), (dict(wu=None), 1),
                       (dict(saved=None), 1), (dict(dwg=None), 1), (dict(dwu=None), 1), (dict(ws=None), 1),
                       (dict(rows=-1), 2), (dict(dys=-1), 2), (dict(xs=-1), 2), (dict(dxs=7), 2), (dict(act=9), 4),
                       (dict(n=need - 1), 4), (dict(n=-1), 4), (dict(ws=ctypes.c_void_p(0x1040)), 4)]:
        assert bwd(**kw) == status, kw
    assert bwd(dx=None, dwg=None, dwu=None, ws=None, n=0) == 0


def join_desc(**over):
    from spatial_transformer_grid_amd.blocks import ResidualNormDesc

    d = ResidualNormDesc()
    vals = dict(dtype=0, param_dtype=0, gate_dtype=0, layer=0, rows=6, cols=8, gate_rows=3, epsilon=1e-5,
                residual_scale=1.0)
    for n in ("x", "branch", "h", "y", "dh", "dy", "dx", "dbranch"):
        vals[n + "_stride"] = 8
    vals.update(over)
    for n, v in vals.items():
        setattr(d, n, v)
    return ctypes.byref(d)


BAD_JOINS = [(dict(dtype=3), 3), (dict(dtype=1, param_dtype=2, gate_dtype=1), 3),
             (dict(dtype=1, param_dtype=1, gate_dtype=2), 3), (dict(rows=-1), 2), (dict(cols=-1), 2), (dict(cols=0), 2),
             (dict(gate_rows=-1), 2), (dict(gate_rows=4), 2), (dict(x_stride=-1), 2), (dict(branch_stride=-8), 2),
             (dict(epsilon=-1.0), 4), (dict(epsilon=math.nan), 4), (dict(epsilon=math.inf), 4),
             (dict(residual_scale=math.inf), 4), (dict(residual_scale=math.nan), 4), (dict(layer=2), 4),
             (dict(cols=16385, h_stride=20000, y_stride=20000, dx_stride=20000, dbranch_stride=20000), 6),
             (dict(rows=2 ** 31, gate_rows=0), 6)]


def test_residual_norm_refuses(tk):
    lib = tk.token_lib()

    def fwd(d, x=FAKE, f=FAKE, m=FAKE, w1=FAKE, b1=FAKE, w2=FAKE, b2=FAKE, h=FAKE, y=FAKE, stats=None):
        return lib.gs_residual_norm(d, x, f, m, w1, b1, w2, b2, h, y, stats, None)

    def bwd(d, dh=FAKE, dy=FAKE, x=FAKE, f=FAKE, m=FAKE, w1=FAKE, b1=FAKE, w2=FAKE, stats=FAKE, dx=FAKE, df=FAKE,
            dm=FAKE, dw1=FAKE, db1=FAKE, dw2=FAKE, db2=FAKE, ws=FAKE, n=1 << 20):
        return lib.gs_residual_norm_backward(d, dh, dy, x, f, m, w1, b1, w2, stats, dx, df, dm, dw1, db1, dw2, db2, ws, n,
                                             None)

    size = lib.gs_residual_norm_backward_workspace_size
    for over, status in BAD_JOINS:
        d = join_desc(**over)
        assert fwd(d) == status and bwd(d) == status and size_of(size, d) == -status, over
    assert fwd(join_desc(h_stride=7)) == 2 and fwd(join_desc(y_stride=7)) == 2
    for n in ("dh_stride", "dy_stride"):
        assert bwd(join_desc(**{n: -1})) == 2
    for n in ("dx_stride", "dbranch_stride"):
        assert bwd(join_desc(**{n: 7})) == 2
    assert fwd(None) == 1 and bwd(None) == 1 and size(join_desc(), None) == 1
    for kw in ("x", "f", "m", "h", "y"):
        assert fwd(join_desc(), **{kw: None}) == 1, kw
    assert fwd(join_desc(), w1=None) == 1 and fwd(join_desc(), w2=None) == 1      # a bias without its scale
    assert fwd(join_desc(), stats=ctypes.c_void_p(0x1004)) == 4
    for kw in ("dy", "x", "f", "m", "stats", "dx", "df", "ws", "w1", "w2"):
        assert bwd(join_desc(), **{kw: None}) == 1, kw
    assert bwd(join_desc(gate_rows=0)) == 1                                        # a gradient of no gate
    need = size_of(size, join_desc())
    assert need > 0
    assert bwd(join_desc(), n=64) == 4 and bwd(join_desc(), n=-1) == 4
    assert bwd(join_desc(), ws=ctypes.c_void_p(0x1010)) == 4 and bwd(join_desc(), stats=ctypes.c_void_p(0x1008)) == 4
    empty = join_desc(rows=0, gate_rows=0)
    assert fwd(empty, *[None] * 9) == 0
    assert bwd(empty, *[None] * 16, ws=None, n=0) == 0


def scan_desc(**over):
    from spatial_transformer_grid_amd.blocks import RecurrenceDesc

    d = RecurrenceDesc()
    vals = dict(dtype=0, batch=2, length=5, channels=8)
    for n in ("x", "g", "y", "dy", "dx", "dg"):
        vals[n + "_stride"] = (40, 8)
    vals.update(over)
    for n, v in vals.items():
        setattr(d, n, (ctypes.c_int64 * 2)(*v) if isinstance(v, tuple) else v)
    return ctypes.byref(d)


def test_gated_recurrence_refuses(tk):
    lib = tk.token_lib()

    def fwd(d, x=FAKE, g=FAKE, y=FAKE, ws=None, n=0):
        return lib.gs_gated_recurrence(d, x, g, None, None, y, None, None, ws, n, None)

    def bwd(d, dy=FAKE, x=FAKE, g=FAKE, saved=FAKE, dx=FAKE, dg=FAKE, ws=None, n=0):
        return lib.gs_gated_recurrence_backward(d, dy, x, g, saved, None, None, dx, dg, None, ws, n, None)

    sizes = (lib.gs_gated_recurrence_workspace_size, lib.gs_gated_recurrence_backward_workspace_size)
    for over, status in [(dict(dtype=3), 3), (dict(batch=-1), 2), (dict(length=-1), 2), (dict(channels=-1), 2),
                         (dict(x_stride=(-1, 8)), 2), (dict(g_stride=(40, -8)), 2), (dict(length=2 ** 29 + 1), 6),
                         (dict(channels=2 ** 22 + 1), 6), (dict(batch=2 ** 30 + 1), 6),
                         (dict(batch=2 ** 16, channels=2 ** 15), 6), (dict(batch=2 ** 22, channels=1), 6),
                         (dict(x_stride=(0, 2 ** 23)), 6), (dict(dtype=2, g_stride=(0, 2 ** 24)), 6)]:
        d = scan_desc(**over)
        assert fwd(d) == status and bwd(d) == status, over
        assert [size_of(s, d) for s in sizes] == [-status] * 2, over
    for s in ((7, 8), (40, 7)):
        assert fwd(scan_desc(y_stride=s)) == 2
        assert bwd(scan_desc(dx_stride=s)) == 2 and bwd(scan_desc(dg_stride=s)) == 2
    assert bwd(scan_desc(dy_stride=(-1, 0))) == 2
    assert fwd(None) == 1 and bwd(None) == 1
    for kw in ("x", "g", "y"):
        assert fwd(scan_desc(), **{kw: None}) == 1
    for kw in ("dy", "x", "g", "saved", "dx", "dg"):
        assert bwd(scan_desc(), **{kw: None}) == 1
    for call in (fwd, bwd):
        assert call(scan_desc(), n=-1) == 4 and call(scan_desc(), ws=ctypes.c_void_p(0x1010), n=64) == 4
        assert call(scan_desc(batch=0), *[None] * 3) == 0 and call(scan_desc(channels=0), *[None] * 3) == 0
    for s in sizes:
        assert s(scan_desc(), None) == 1
        assert size_of(s, scan_desc()) == 0
        assert size_of(s, scan_desc(batch=1, length=65536)) > 0                    # few channels, many tokens


def test_binding_refuses(tk):
    import spatial_transformer_grid_amd as gs

    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError):
        gs.gated_linear(x, w, w)
    with pytest.raises(ValueError):
        gs.residual_norm(x, x, torch.ones(8))
    with pytest.raises(ValueError):
        gs.gated_recurrence(x[None], x[None])
    with pytest.raises(ValueError):
        gs.gated_recurrence(x, x)
    for bad in ("swish", 0, None):
        with pytest.raises(ValueError):
            gs.blocks._named(bad, gs.blocks.ACTIVATIONS, "activation")
    assert set(gs.blocks.__all__) == {n for n in dir(gs) if n.startswith(("gated_", "residual_norm"))}


def test_every_call_with_a_stream_hands_over(monkeypatch):
    import inspect

    from spatial_transformer_grid_amd import blocks

    seen = []
    monkeypatch.setattr(blocks, "_on_stream", lambda *a, **kw: seen.append((a, kw)))
    for name in blocks.__all__:
        c = getattr(blocks, name)
        sig = inspect.signature(c).parameters
        given = {n: "value of " + n for n in sig}
        c(**given)
        a, kw = seen.pop()
        assert a[:2] == (given.pop("stream"), c)
        # every argument is handed on under its own name
        assert inspect.signature(c).bind(*a[2:], **kw).arguments == given
