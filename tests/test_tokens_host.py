"""The token operators without a GPU: the 64-bit reference against published
values, closed forms, torch and differences; bucket borders; the C ABI's
exports, descriptor layout and refusals (every call here fails validation or
has nothing to do)."""

import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import token_reference as ref
from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "gsample_tokens.h")
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails before


@pytest.fixture(scope="module")
def tk():
    from spatial_transformer_grid_amd import _binding, _tokens

    if not os.path.exists(_binding.LIB_PATH):
        from spatial_transformer_grid_amd import build

        build.build()
    return _tokens


# ------------------------------------------------------------- reference

def test_generator_known_answers():
    """The answers published with the generator for Philox4x32-10."""
    def words(c, k):
        return [int(x[0]) for x in ref.philox([np.array([v], dtype=np.uint64) for v in c], k)]

    assert words((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert words((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_reference_dropout_share_and_mean():
    x = torch.ones(200000, dtype=torch.float64)
    for ratio in (0.0, 0.1, 0.5, 0.9):
        y = ref.dropout(x, ratio, 7, 1)
        p = math.floor(ratio * 65536 + 0.5) / 65536
        # five standard deviations of a binomial share
        assert abs((y == 0).double().mean() - p) <= 5 * math.sqrt(p * (1 - p) / len(x)) + 1e-12
        assert set(y.unique().tolist()) <= {0.0, 65536 / (65536 - p * 65536)}


def test_reference_layer_norm_is_torchs():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 33, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(33, generator=g, dtype=torch.float64, requires_grad=True)
    b = torch.randn(33, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(5, 33, generator=g, dtype=torch.float64)
    y = torch.nn.functional.layer_norm(x, (33,), w, b, 1e-5)
    y.backward(dy)
    assert torch.allclose(ref.layer_norm(x.detach(), w.detach(), b.detach(), 1e-5)[0], y, atol=1e-12)
    got = ref.layer_norm_backward(dy, x.detach(), w.detach(), 1e-5)
    for a, t in zip(got, (x, w, b)):
        assert torch.allclose(a, t.grad, atol=1e-11)


def reference_case(**over):
    c = dict(B=2, H=4, Hkv=2, Lq=5, Lk=9, D=3, causal=0, lengths=(9, 4), buckets=8, distance=6, bidirectional=1,
             first=0, ratio=0.25)
    c.update(over)
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    q, k, v = r(c["B"], c["H"], c["Lq"], c["D"]), r(c["B"], c["Hkv"], c["Lk"], c["D"]), r(
        c["B"], c["Hkv"], c["Lk"], c["D"])
    table, do = r(c["buckets"], c["H"]), r(c["B"], c["H"], c["Lq"], c["D"])
    def call(q, k, v, table, do=None):
        return ref.attention(q, k, v, 0.6, c["causal"], torch.tensor(c["lengths"]), table, c["distance"],
                             c["bidirectional"], c["first"], c["ratio"], 99, 4, do)
    return q, k, v, table, do, call


@pytest.mark.parametrize("over", [{}, dict(causal=1, first=2, bidirectional=0), dict(lengths=(0, 9)),
                                  dict(causal=1, first=-3, ratio=0.0)])
def test_reference_gradients_against_differences(over):
    """Central differences of sum(o * dO) in every input element."""
    q, k, v, table, do, call = reference_case(**over)
    got = call(q, k, v, table, do)
    inputs = {"dq": q, "dk": k, "dv": v, "dtable": table}
    h = 1e-5
    for name, t in inputs.items():
        num = torch.zeros_like(t)
        for i in range(t.numel()):
            vals = []
            for sign in (1, -1):
                moved = {n: x.clone() for n, x in inputs.items()}
                moved[name].view(-1)[i] += sign * h
                o = call(moved["dq"], moved["dk"], moved["dv"], moved["dtable"])["o"][0]
                vals.append((o * do).sum())
            num.view(-1)[i] = (vals[0] - vals[1]) / (2 * h)
        # h^2 times third derivatives of order one, rounding 1e-16 / h
        assert torch.allclose(got[name][0], num, atol=1e-7), name


def test_reference_attention_without_extras_is_softmax():
    q, k, v, table, do, _ = reference_case()
    got = ref.attention(q, k, v, 0.6, 0, None, None, 6, 1, 0, 0.0, 0, 0)["o"][0]
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    assert torch.allclose(got, torch.softmax(q @ kk.transpose(-1, -2) * 0.6, -1) @ vv, atol=1e-13)


# --------------------------------------------------------------- buckets

@pytest.mark.parametrize("num,distance,both", [(32, 128, 1), (32, 128, 0), (4, 40, 1), (2, 2, 0), (8, 6, 1),
                                               (64, 256, 1), (320, 800, 1), (320, 800, 0), (2, 1000, 0),
                                               (32, 1000, 0), (3, 7, 0), (512, 1023, 0), (32, 9, 1)])
def test_buckets_match_whole_number_borders(tk, num, distance, both):
    rels = list(range(-1100, 1101)) + [-(2 ** 40), 2 ** 40, -(2 ** 63), 2 ** 63 - 1]
    want = ref.bucket(np.array(rels, dtype=object).clip(-5000, 5000).astype(np.int64), num, distance, both)
    assert [tk.relative_bucket(r, num, distance, both) for r in rels] == want.tolist()


def test_buckets_by_hand(tk):
    """32 buckets up to 128, both directions: 8 single distances a side, then
    borders at 8 * 2^(j/2): 8, 11.3, 16, 22.6, 32, 45.3, 64, 90.5."""
    for d, b in [(0, 0), (1, 1), (7, 7), (8, 8), (11, 8), (12, 9), (15, 9), (16, 10), (22, 10), (23, 11), (31, 11),
                 (32, 12), (45, 12), (46, 13), (63, 13), (64, 14), (90, 14), (91, 15), (128, 15), (100000, 15)]:
        assert tk.relative_bucket(-d, 32, 128, 1) == b
        assert tk.relative_bucket(d, 32, 128, 1) == (b + 16 if d else 0)
        assert tk.relative_bucket(d, 32, 128, 0) == 0


def test_buckets_refused(tk):
    from spatial_transformer_grid_amd import GSError

    for args, status in [((0, 1, 8, 0), 4), ((0, 513, 8, 0), 4), ((0, 5, 8, 1), 4), ((0, 2, 8, 1), 4),
                         ((0, 32, 8, 1), 4), ((0, 32, 16, 0), 4), ((0, 32, 8, 2), 4), ((0, 32, 100000, 1), 6)]:
        with pytest.raises(GSError) as e:
            tk.relative_bucket(*args)
        assert e.value.status == status, args


# ------------------------------------------------------------------- ABI

def test_exports_and_signatures(tk):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s*(gs_\w+)\s*\(", text, flags=re.M))
    assert names == set(tk.TOKEN_SIGNATURES)
    for n in names:
        assert hasattr(tk.token_lib(), n), n
        args = re.search(r"\b%s\s*\((.*?)\);" % n, text, flags=re.S).group(1)
        assert len(args.split(",")) == len(tk.TOKEN_SIGNATURES[n][0]), n


def test_descriptor_layout(tk, tmp_path):
    fields = [f[0] for f in tk.AttentionDesc._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gsample_tokens.h"\nint main(void) {\n' +
                   "".join('printf("%%zu\\n", offsetof(gs_attention_desc, %s));\n' % f for f in fields) +
                   'printf("%zu\\n", sizeof(gs_attention_desc)); return 0; }\n')
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe],
                   check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(tk.AttentionDesc, f).offset for f in fields] + [ctypes.sizeof(tk.AttentionDesc)]


def desc(tk, **over):
    d = tk.AttentionDesc()
    vals = dict(dtype=0, table_dtype=0, batch=2, q_heads=4, kv_heads=2, q_len=5, kv_len=7, head_dim=8, scale=0.5,
                causal=0, q_from_end=0, q_position=0, num_buckets=8, max_distance=16, bidirectional=1, ratio=0.1)
    for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv"):
        vals[n + "_stride"] = (ctypes.c_int64 * 3)(280, 56, 8)
    vals.update(over)
    for n, v in vals.items():
        setattr(d, n, v)
    return d


BAD_DESCRIPTORS = [
    (dict(dtype=3), 3), (dict(dtype=-1), 3), (dict(table_dtype=1), 3), (dict(batch=-1), 2), (dict(q_len=-1), 2),
    (dict(kv_len=-1), 2), (dict(q_heads=3), 2), (dict(kv_heads=0), 2), (dict(head_dim=0), 2),
    (dict(k_stride=(ctypes.c_int64 * 3)(1, -1, 8)), 2), (dict(scale=math.nan), 4), (dict(scale=math.inf), 4),
    (dict(causal=2), 4), (dict(q_from_end=-1), 4), (dict(ratio=-0.1), 4), (dict(ratio=1.0), 4),
    (dict(ratio=0.999999), 4), (dict(ratio=math.nan), 4), (dict(num_buckets=1), 4), (dict(num_buckets=7), 4),
    (dict(num_buckets=-4), 4), (dict(num_buckets=514), 4), (dict(max_distance=2), 4), (dict(bidirectional=3), 4),
    (dict(max_distance=10 ** 6), 6), (dict(head_dim=129), 6), (dict(q_len=2 ** 29 + 1), 6),
    (dict(kv_len=2 ** 29 + 1), 6), (dict(q_position=2 ** 29 + 1), 6), (dict(q_position=-(2 ** 29) - 1), 6),
    (dict(batch=2 ** 30), 6), (dict(q_heads=2 ** 22, kv_heads=2 ** 22), 6), (dict(q_heads=0, kv_heads=2 ** 30), 6),
]


@pytest.mark.parametrize("over,status", BAD_DESCRIPTORS)
def test_attention_refuses_descriptors(tk, over, status):
    lib, need = tk.token_lib(), ctypes.c_int64(-1)
    d = ctypes.byref(desc(tk, **over))
    assert lib.gs_attention(d, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, None, 0, None) == status
    assert lib.gs_attention_workspace_size(d, ctypes.byref(need)) == status
    assert lib.gs_attention_backward(d, *[FAKE] * 6, None, *[FAKE] * 5, ctypes.c_void_p(4096), 1 << 20,
                                     None) == status
    assert lib.gs_attention_backward_workspace_size(d, ctypes.byref(need)) == status
    assert need.value == -1


def test_attention_refuses_pointers_and_workspaces(tk):
    lib, need = tk.token_lib(), ctypes.c_int64(0)
    d = ctypes.byref(desc(tk))
    assert lib.gs_attention(None, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, None, 0, None) == 1
    for missing in (0, 1, 2, 4, 5):
        a = [FAKE, FAKE, FAKE, None, FAKE, FAKE]
        a[missing] = None
        assert lib.gs_attention(d, *a, None, None, 0, None) == 1
    assert lib.gs_attention(d, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, ctypes.c_void_p(0x1010), 64, None) == 4
    assert lib.gs_attention(d, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, -1, None) == 4
    assert lib.gs_attention_workspace_size(d, None) == 1
    assert lib.gs_attention_backward_workspace_size(d, ctypes.byref(need)) == 0 and need.value > 0
    ok = [FAKE] * 6 + [None] + [FAKE] * 5
    for missing in (0, 1, 2, 3, 4, 5, 7, 8, 9, 10):
        a = list(ok)
        a[missing] = None
        assert lib.gs_attention_backward(d, *a, FAKE, need.value, None) == 1, missing
    assert lib.gs_attention_backward(d, *ok, None, 0, None) == 1
    assert lib.gs_attention_backward(d, *ok, FAKE, need.value - 1, None) == 4
    assert lib.gs_attention_backward(d, *ok, ctypes.c_void_p(0x1008), need.value, None) == 4
    assert lib.gs_attention_backward(d, *ok, FAKE, -1, None) == 4


def test_empty_calls_need_nothing(tk):
    lib = tk.token_lib()
    for over in (dict(batch=0), dict(q_len=0), dict(q_heads=0)):
        d = ctypes.byref(desc(tk, **over))
        assert lib.gs_attention(d, *[None] * 7, None, 0, None) == 0
    assert lib.gs_layer_norm(None, 0, 0, 8, 8, None, None, 0, 1e-5, None, 8, None, None, None) == 0
    assert lib.gs_dropout(None, 0, 0, None, 0.5, 1, 1, None, None) == 0


def test_layer_norm_refuses(tk):
    lib = tk.token_lib()

    def fwd(dtype=0, rows=4, cols=8, xs=8, scale=FAKE, pd=0, eps=1e-5, x=FAKE, y=FAKE, ys=8):
        return lib.gs_layer_norm(x, dtype, rows, cols, xs, scale, None, pd, eps, y, ys, None, None, None)

    for kw, status in [(dict(rows=-1), 2), (dict(cols=-1), 2), (dict(cols=0), 2), (dict(xs=-8), 2), (dict(ys=7), 2),
                       (dict(dtype=3), 3), (dict(dtype=1, pd=2), 3), (dict(pd=3), 3), (dict(eps=-1.0), 4),
                       (dict(eps=math.nan), 4), (dict(eps=math.inf), 4), (dict(cols=2 ** 24 + 1, ys=2 ** 25), 6),
                       (dict(rows=2 ** 31), 6), (dict(x=None), 1), (dict(y=None), 1), (dict(scale=None), 1)]:
        assert fwd(**kw) == status, kw

    def bwd(dy=FAKE, x=FAKE, rows=4, dxs=8, scale=FAKE, mean=FAKE, inv=FAKE, dx=FAKE, ds=FAKE, db=FAKE, ws=FAKE,
            n=None):
        need = ctypes.c_int64(0)
        assert lib.gs_layer_norm_backward_workspace_size(4, 8, ctypes.byref(need)) == 0 and need.value > 0
        return lib.gs_layer_norm_backward(dy, x, 0, rows, 8, 8, 8, scale, 0, mean, inv, dx, dxs, ds, db, ws,
                                          need.value if n is None else n, None)

    for kw, status in [(dict(dy=None), 1), (dict(x=None), 1), (dict(scale=None), 1), (dict(mean=None), 1),
                       (dict(inv=None), 1), (dict(dx=None), 1), (dict(ds=None), 1), (dict(db=None), 1),
                       (dict(ws=None), 1), (dict(n=8), 4), (dict(n=-1), 4), (dict(ws=ctypes.c_void_p(0x1010)), 4),
                       (dict(rows=-1), 2), (dict(dxs=3), 2)]:
        assert bwd(**kw) == status, kw
    assert lib.gs_layer_norm_backward_workspace_size(4, 8, None) == 1


def test_dropout_refuses(tk):
    lib = tk.token_lib()
    for a, status in [((None, 0, 8, None, 0.5, 1, 1, FAKE, None), 1), ((FAKE, 0, 8, None, 0.5, 1, 1, None, None), 1),
                      ((FAKE, 0, -1, None, 0.5, 1, 1, FAKE, None), 2), ((FAKE, 3, 8, None, 0.5, 1, 1, FAKE, None), 3),
                      ((FAKE, 0, 8, None, 1.0, 1, 1, FAKE, None), 4), ((FAKE, 0, 8, None, -0.1, 1, 1, FAKE, None), 4),
                      ((FAKE, 0, 8, None, math.nan, 1, 1, FAKE, None), 4),
                      ((FAKE, 0, 2 ** 40 + 1, None, 0.5, 1, 1, FAKE, None), 6)]:
        assert lib.gs_dropout(*a) == status, a


def test_binding_refuses_host_tensors(tk):
    x, q = torch.zeros(4, 8), torch.zeros(1, 2, 3, 8)
    with pytest.raises(ValueError):
        tk.layer_norm(x, torch.ones(8))
    with pytest.raises(ValueError):
        tk.dropout(x, 0.1, 1)
    with pytest.raises(ValueError):
        tk.attention(q, q, q)
    with pytest.raises(ValueError):
        tk.attention(q[0], q, q)
