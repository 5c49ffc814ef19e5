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
