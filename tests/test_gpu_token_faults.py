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
