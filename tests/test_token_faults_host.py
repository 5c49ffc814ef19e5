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
            def ExternalStream(handle, device):
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


@pytest.mark.parametrize("given", ["stream", "handle", "current", None])
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

    stream = {"stream": FakeStream(2, log), "handle": 2, "current": fake.now, None: 1}[given]
    assert _binding._on_stream(stream, call, x, 3, workspace=ws) == (y, None, z)
    if given in ("current", None):
        assert log == [("call", 1)]
    else:
        assert log == [("wait", 2, 1), ("record", "x", 2), ("record", "ws", 2), ("call", 2), ("record", "y", 1),
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


# ---------------------------------------------------------------- scratch

def test_scratch_must_be_contiguous_gpu_memory(tk):  # noqa: F811
    """Scratch in host memory, on another GPU or with gaps is refused, by the token calls and the older ones."""
    class Scratch(torch.Tensor):
        @staticmethod
        def of(t, device):
            t = t.as_subclass(Scratch)
            t.place = torch.device(device)
            return t

        is_cuda = property(lambda self: self.place.type == "cuda")
        device = property(lambda self: self.place)

    here = torch.device("cuda:0")
    flat = torch.zeros(512, dtype=torch.uint8)
    for bad in (flat, Scratch.of(flat, "cuda:1"), Scratch.of(flat[::2], "cuda:0")):
        with pytest.raises(ValueError):
            tk._workspace(bad, 256, here)
    good = Scratch.of(flat, "cuda:0")
    assert tk._workspace(good, 256, here)[1:] == (flat.data_ptr(), 512)
    assert tk._workspace(flat[:0], 256, here) == (None, None, 0)
