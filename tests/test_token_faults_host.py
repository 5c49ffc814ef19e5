"""Refusals and plans of the token operators that need no GPU: every call here
fails validation, has nothing to do, or asks for a size."""

import ctypes

import pytest
import torch

from test_tokens_host import FAKE, desc, tk  # noqa: F401


def test_backward_without_query_heads_still_has_gradients_to_write(tk):  # noqa: F811
    """dK and dV of key heads that no query head reads are outputs: their pointers are asked for."""
    lib = tk.token_lib()
    d = ctypes.byref(desc(tk, q_heads=0, kv_heads=4))
    assert lib.gs_attention_backward(d, *[None] * 12, None, 0, None) == 1
    for over in (dict(q_heads=0, kv_heads=0), dict(q_heads=0, kv_heads=4, batch=0), dict(q_heads=0, kv_len=0)):
        d = ctypes.byref(desc(tk, **over))
        assert lib.gs_attention_backward(d, *[None] * 12, None, 0, None) == 0, over


# ---------------------------------------------------------------- streams

class FakeStream:
    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))


class FakeTensor:
    is_cuda, device = True, "cuda:0"

    def __init__(self, name, log):
        self.name, self.log = name, log

    def record_stream(self, stream):
        self.log.append(("record", self.name, stream.cuda_stream))


class FakeTorch:
    """As much of torch as a stream's hand-over uses; the current stream has handle 1."""

    Tensor = FakeTensor

    def __init__(self, log):
        torch_ = self

        class cuda:
            Stream = FakeStream

            @staticmethod
            def current_stream(device):
                return torch_.now

            @staticmethod
            def default_stream(device):
                return FakeStream(0, log)

            @staticmethod
            def ExternalStream(handle, device):
                assert handle
                return FakeStream(handle, log)

            @staticmethod
            def stream(s):
                class On:
                    def __enter__(self):
                        self.before, torch_.now = torch_.now, s

                    def __exit__(self, *_):
                        torch_.now = self.before
                return On()

        self.cuda, self.now = cuda, FakeStream(1, log)


@pytest.mark.parametrize("given", ["stream", "handle", "null", "current", None])
def test_stream_argument_hands_memory_over(monkeypatch, given):
    """A call on a named stream starts after the current one, runs with it current (so copies and scratch are its
    own), and inputs and outputs are kept for both."""
    from spatial_transformer_grid_amd import _binding

    log = []
    fake = FakeTorch(log)
    monkeypatch.setattr(_binding, "_torch", lambda: fake)
    x, ws, y, z = (FakeTensor(n, log) for n in ("x", "ws", "y", "z"))

    def call(a, b, workspace=None):
        assert (a, b, workspace) == (x, 3, ws)
        log.append(("call", fake.now.cuda_stream))
        return y, None, z

    stream = {"stream": FakeStream(2, log), "handle": 2, "null": 0, "current": fake.now, None: 1}[given]
    assert _binding._on_stream(stream, call, x, 3, workspace=ws) == (y, None, z)
    if given in ("current", None):
        assert log == [("call", 1)]
    else:
        to = 0 if given == "null" else 2
        assert log == [("wait", to, 1), ("record", "x", to), ("record", "ws", to), ("call", to), ("record", "y", 1),
                       ("record", "z", 1)]
    assert fake.now.cuda_stream == 1


def test_every_call_with_a_stream_hands_over(monkeypatch):
    import inspect

    import spatial_transformer_grid_amd as gsa
    from spatial_transformer_grid_amd import _binding, _tokens

    calls = [getattr(gsa, n) for n in gsa.__all__ if callable(getattr(gsa, n))]
    calls = [c for c in calls if inspect.isfunction(c) and "stream" in inspect.signature(c).parameters]
    assert len(calls) == 12
    seen = []
    for module in (_binding, _tokens):
        monkeypatch.setattr(module, "_on_stream", lambda *a, **kw: seen.append((a, kw)))
    for c in calls:
        sig = inspect.signature(c).parameters
        given = {n: "value of " + n for n in sig}
        c(**given)
        a, kw = seen.pop()
        assert a[:2] == (given.pop("stream"), c)
        # every argument is handed on under its own name
        bound = inspect.signature(c).bind(*a[2:], **kw).arguments
        assert dict(bound) == given


# ------------------------------------------------------ scratch and devices

class Placed(torch.Tensor):
    """A host tensor that says it lies on a device."""

    @staticmethod
    def of(t, device):
        t = t.as_subclass(Placed)
        t.place = torch.device(device)
        return t

    is_cuda = property(lambda self: self.place.type == "cuda")
    device = property(lambda self: self.place)

    def get_device(self):
        return self.place.index if self.is_cuda else -1


def test_scratch_must_be_contiguous_gpu_memory(tk):  # noqa: F811
    """Scratch in host memory, on another GPU or with gaps is refused, by the token calls and the older ones."""
    here = torch.device("cuda:0")
    flat = torch.zeros(512, dtype=torch.uint8)
    for bad in (flat, Placed.of(flat, "cuda:1"), Placed.of(flat[::2], "cuda:0")):
        with pytest.raises(ValueError):
            tk._workspace(bad, 256, here)
    good = Placed.of(flat, "cuda:0")
    assert tk._workspace(good, 256, here)[1:] == (flat.data_ptr(), 512)
    assert tk._workspace(flat[:0], 256, here) == (None, None, 0)


def test_tensors_of_two_gpus_are_refused(tk):  # noqa: F811
    import spatial_transformer_grid_amd as gsa

    def on(i, *shape, dtype=torch.float32):
        return Placed.of(torch.zeros(*shape, dtype=dtype), "cuda:%d" % i)

    q, far, lse = on(0, 1, 2, 3, 8), on(1, 1, 2, 3, 8), on(0, 1, 2, 3)
    x, w, row = on(0, 4, 8), on(0, 8), on(0, 4)
    for call in (lambda: gsa.attention(q, far, q), lambda: gsa.attention(q, q, far),
                 lambda: gsa.attention(q, q, q, kv_lengths=on(1, 1, dtype=torch.int32)),
                 lambda: gsa.attention(q, q, q, table=on(1, 8, 2)), lambda: gsa.attention(q, q, q, out=far),
                 lambda: gsa.attention_backward(far, q, q, q, q, lse),
                 lambda: gsa.attention_backward(q, q, q, q, far, lse),
                 lambda: gsa.attention_backward(q, q, q, q, q, on(1, 1, 2, 3)),
                 lambda: gsa.layer_norm(x, on(1, 8)), lambda: gsa.layer_norm(x, w, on(1, 8)),
                 lambda: gsa.layer_norm(x, w, out=on(1, 4, 8)),
                 lambda: gsa.layer_norm_backward(on(1, 4, 8), x, w, row, row),
                 lambda: gsa.layer_norm_backward(x, x, w, on(1, 4), row),
                 lambda: gsa.layer_norm_backward(x, x, w, row, on(1, 4)),
                 lambda: gsa.dropout(x, 0.1, 1, residual=on(1, 4, 8)), lambda: gsa.dropout(x, 0.1, 1, out=on(1, 4, 8)),
                 lambda: gsa.affine_grid(on(0, 1, 2, 3), (1, 1, 2, 2), out=on(1, 1, 2, 2, 2)),
                 lambda: gsa.grid_sample(q, on(1, 1, 3, 3, 2)), lambda: gsa.resize(q, sizes=(1, 2, 3, 8), out=far),
                 lambda: gsa.affine_grid_sample_fused(on(1, 1, 2, 3), q, (3, 8)),
                 lambda: gsa.deform_conv(q, on(1, 2, 2, 1, 1), on(0, 1, 2, 3, 8)),
                 lambda: gsa.deform_conv(q, on(0, 2, 2, 1, 1), on(1, 1, 2, 3, 8))):
        with pytest.raises(ValueError, match="GPU"):
            call()


# ---------------------------------------------------------------- outputs

@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("name", ["o", "dq", "dk", "dv"])
def test_outputs_with_overlapping_rows_are_refused(tk, name, axis):  # noqa: F811
    """A broadcast output, or one whose rows begin inside the row before, along any axis; an axis of one element
    takes any stride, and so does every axis of a tensor without elements."""
    lib, need = tk.token_lib(), ctypes.c_int64(0)
    def strides(value):
        s = [280, 56, 8]
        s[axis] = value
        return {name + "_stride": (ctypes.c_int64 * 3)(*s)}
    def statuses(**over):
        d = ctypes.byref(desc(tk, **over))
        return (lib.gs_attention_workspace_size(d, ctypes.byref(need)),
                lib.gs_attention_backward_workspace_size(d, ctypes.byref(need)))
    forward = name == "o"
    for bad in (0, 1, 7):
        got = statuses(**strides(bad))
        assert got == ((2, 0) if forward else (0, 2)), bad
        d = ctypes.byref(desc(tk, **strides(bad)))
        if forward:
            assert lib.gs_attention(d, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, None, 0, None) == 2
        else:
            assert lib.gs_attention_backward(d, *[FAKE] * 6, None, *[FAKE] * 5, FAKE, 1 << 20, None) == 2
    one = [dict(batch=1), dict(q_heads=1, kv_heads=1), dict(q_len=1, kv_len=1)][axis]
    assert statuses(**strides(0), **one) == (0, 0)
    assert statuses(**strides(0), batch=0) == (0, 0)
    assert statuses(**strides(8)) == (0, 0)


# ---------------------------------------------------------------- buckets

@pytest.mark.parametrize("num,distance,both", [
    (21, 1006, 0), (42, 1006, 1),                    # the border whose two sides are closest to each other
    (32, 128, 1), (16, 512, 0), (6, 24, 1), (64, 1000, 0), (511, 1000, 0), (512, 1024, 1), (24, 96, 0), (5, 32, 0),
    (3, 1 << 20, 0), (2, 2 ** 31 - 1, 0), (4, 2 ** 31 - 1, 1), (7, 4000, 0), (20, 640, 1), (100, 800, 0)])
def test_bucket_borders_where_both_sides_are_close_or_equal(tk, num, distance, both):  # noqa: F811
    import numpy as np

    import token_reference as ref

    d = np.arange(-1100, 1101)
    assert [tk.relative_bucket(int(r), num, distance, both) for r in d] == ref.bucket(d, num, distance, both).tolist()


# ---------------------------------------------------------- launch limits

def test_grids_that_no_launch_takes_are_refused(tk):  # noqa: F811
    """2^24 blocks of 256 threads are 2^32 threads: the first size that a launch refuses."""
    lib, need = tk.token_lib(), ctypes.c_int64(0)
    strides = {n + "_stride": (ctypes.c_int64 * 3)(1 << 24, 8, 8) for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv")}
    heads = 1 << 20
    for over, status in [(dict(batch=16, q_heads=heads, kv_heads=heads), 6),
                         (dict(batch=16, q_heads=heads - 1, kv_heads=heads - 1), 0),
                         (dict(batch=1, q_heads=heads, kv_heads=heads, q_len=512, kv_len=1), 6),
                         (dict(batch=1, q_heads=heads, kv_heads=heads, q_len=1, kv_len=481), 6),
                         (dict(batch=1, q_heads=heads, kv_heads=heads, q_len=480, kv_len=480), 0)]:
        d = ctypes.byref(desc(tk, **{**dict(q_len=1, kv_len=1, **strides), **over}))
        assert lib.gs_attention_workspace_size(d, ctypes.byref(need)) == status, over
        assert lib.gs_attention_backward_workspace_size(d, ctypes.byref(need)) == status, over
    d = ctypes.byref(desc(tk, batch=1, q_heads=1 << 15, kv_heads=1 << 15, q_len=1, kv_len=1, num_buckets=512,
                          max_distance=1000, **strides))
    assert lib.gs_attention_backward(d, *[FAKE] * 6, None, *[FAKE] * 5, None, 0, None) == 6
    # without dtable nothing is summed for it
    assert lib.gs_attention_backward(d, *[FAKE] * 6, None, FAKE, FAKE, FAKE, FAKE, None, None, 0, None) == 1


@pytest.mark.parametrize("over", [dict(r=1 << 63), dict(num_buckets=(1 << 32) + 32), dict(max_distance=(1 << 32) + 128),
                                  dict(bidirectional=1 << 32)])
def test_numbers_that_a_field_cuts_are_refused(tk, over):  # noqa: F811
    good = dict(r=-20, num_buckets=32, max_distance=128, bidirectional=1)
    assert tk.relative_bucket(**good) == 10
    with pytest.raises(ValueError):
        tk.relative_bucket(**{**good, **over})
    if "max_distance" in over or "bidirectional" in over:
        q = Placed.of(torch.zeros(1, 2, 3, 8), "cuda:0")
        table = Placed.of(torch.zeros(32, 2), "cuda:0")
        for wrong in (over, dict(causal=1 << 32), dict(q_position=1 << 64)):
            with pytest.raises(ValueError, match="bits"):
                tk._attention_inputs(q, q, q, **{**dict(
                    scale=None, causal=0, kv_lengths=None, table=table, max_distance=128, bidirectional=1, q_position=0,
                    ratio=0.0, seed=0, call=0), **wrong})


# ------------------------------------------------------------------ plans

# B, H, Hkv, Lq, Lk, D: 64 blocks of 128 keys whose (head, query tile) pairs are split over parts
SPLIT_128 = [(4, 64, 16, 520, 33, 64), (4, 32, 8, 520, 201, 128), (2, 64, 32, 1100, 77, 48), (8, 8, 8, 1030, 65, 128)]


@pytest.mark.parametrize("shape", SPLIT_128)
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_split_of_128_key_blocks_is_planned(tk, shape, dtype):  # noqa: F811
    """The workspace holds four numbers a query (five with a table), the table's sums of (blocks of 128 keys) x parts,
    and the parts of dK and dV."""
    B, H, Hkv, Lq, Lk, D = shape
    lib, need = tk.token_lib(), ctypes.c_int64(0)
    def size(buckets):
        d = ctypes.byref(desc(tk, dtype=dtype, table_dtype=0, batch=B, q_heads=H, kv_heads=Hkv, q_len=Lq, kv_len=Lk,
                              head_dim=D, num_buckets=buckets, **{n + "_stride": (ctypes.c_int64 * 3)(1 << 30, 1 << 20, 128)
                                                                  for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv")}))
        assert lib.gs_attention_backward_workspace_size(d, ctypes.byref(need)) == 0
        return need.value
    rounded = lambda n: (n + 255) // 256 * 256
    queries = B * H * ((Lq + 63) // 64) * 64
    sums = size(0) - queries * 16
    parts, rest = divmod(sums, rounded(B * Hkv * Lk * 2 * D * 4))
    assert rest == 0 and parts >= 2
    assert size(8) - size(0) == rounded(B * H * ((Lk + 127) // 128) * parts * 8 * 4) + queries * 4
