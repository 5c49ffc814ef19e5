"""ctypes binding of libgsample's token operators (include/gsample_tokens.h).

Argument marshalling only, as in _binding: layer normalisation, dropout and
attention with a relative position bias, forward and backward.  Tensors may be
strided where the library takes strides; the last axis is made contiguous.
The functions take part in no autograd graph: results are detached, and a
training step calls the _backward functions itself.
"""

from __future__ import annotations

import ctypes
import math

from ._binding import (GS_F32, GS_OK, _check, _device_tensor, _I, _on_gpu, _on_stream, _P, _ptr, _scratch, _stream,
                       _torch, dtype_code)
from ._binding import lib as _library

_I64 = ctypes.c_int64
_F = ctypes.c_float
_U32 = ctypes.c_uint32
_U64 = ctypes.c_uint64
_S3 = ctypes.c_int64 * 3
_PI64 = ctypes.POINTER(ctypes.c_int64)


class AttentionDesc(ctypes.Structure):
    """gs_attention_desc"""

    _fields_ = ([("dtype", _I), ("table_dtype", _I)]
                + [(n, _I64) for n in ("batch", "q_heads", "kv_heads", "q_len", "kv_len", "head_dim")]
                + [(n + "_stride", _S3) for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv")]
                + [("scale", _F), ("causal", _I), ("q_from_end", _I), ("q_position", _I64),
                   ("num_buckets", _I), ("max_distance", _I), ("bidirectional", _I), ("ratio", _F),
                   ("call", _U32), ("seed", _U64)])


_PDESC = ctypes.POINTER(AttentionDesc)
_MASK32, _MASK64 = 2 ** 32 - 1, 2 ** 64 - 1

# C entry points and their argument types (mirrors include/gsample_tokens.h)
TOKEN_SIGNATURES = {
    "gs_layer_norm": ([_P, _I, _I64, _I64, _I64, _P, _P, _I, _F, _P, _I64, _P, _P, _P], _I),
    "gs_layer_norm_backward": ([_P, _P, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _P, _I64, _P, _P,
                                _P, _I64, _P], _I),
    "gs_layer_norm_backward_workspace_size": ([_I64, _I64, _PI64], _I),
    "gs_dropout": ([_P, _I, _I64, _P, _F, _U64, _U32, _P, _P], _I),
    "gs_relative_bucket": ([_I64, _I, _I, _I, ctypes.POINTER(_I)], _I),
    "gs_attention": ([_PDESC, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P], _I),
    "gs_attention_workspace_size": ([_PDESC, _PI64], _I),
    "gs_attention_backward": ([_PDESC] + [_P] * 13 + [_I64, _P], _I),
    "gs_attention_backward_workspace_size": ([_PDESC, _PI64], _I),
    # (blocks; descriptors are passed by reference)
    "gs_gated_linear": ([_P, _I] + [_I64] * 4 + [_P, _P, _I, _P, _I64, _P, _P, _I64, _P], _I),
    "gs_gated_linear_workspace_size": ([_I, _I64, _I64, _I64, _PI64], _I),
    "gs_gated_linear_backward": ([_P, _P, _I] + [_I64] * 5 + [_P, _P, _I, _P, _P, _I64, _P, _P, _P, _I64, _P], _I),
    "gs_gated_linear_backward_workspace_size": ([_I, _I64, _I64, _I64, _PI64], _I),
    "gs_residual_norm": ([_P] * 12, _I),
    "gs_residual_norm_backward": ([_P] * 18 + [_I64, _P], _I),
    "gs_residual_norm_backward_workspace_size": ([_P, _PI64], _I),
    "gs_gated_recurrence": ([_P] * 9 + [_I64, _P], _I),
    "gs_gated_recurrence_workspace_size": ([_P, _PI64], _I),
    "gs_gated_recurrence_backward": ([_P] * 11 + [_I64, _P], _I),
    "gs_gated_recurrence_backward_workspace_size": ([_P, _PI64], _I),
}

_typed = None


def token_lib():
    """The loaded libgsample with the token entry points' argument types set."""
    global _typed
    if _typed is None:
        handle = _library()
        for name, (args, res) in TOKEN_SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _typed = handle
    return _typed


def _tensor(t, name, device=None, dtype=None, shape=None):
    """`t` on the GPU (number `device`) with a contiguous last axis, its type and shape checked."""
    _on_gpu(t, name, device)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must have element type %s" % (name, dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    return t if t.dim() == 0 or t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


def _like(t):
    """A new tensor laid out like `t` (a broadcast axis or a gap is not kept), its last axis contiguous."""
    torch = _torch()
    if 0 not in t.stride():
        new = torch.empty_like(t)
        if new.shape[-1] <= 1 or new.stride(-1) == 1:
            return new
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _output(out, like, dense):
    """`out` checked, or a new tensor: contiguous where `dense`, else laid out like `like`."""
    if out is None:
        if not dense:
            return _like(like)
        torch = _torch()
        return torch.empty_like(like) if like.is_contiguous() else torch.empty(
            like.shape, dtype=like.dtype, device=like.device)
    if out.get_device() != like.get_device() or out.shape != like.shape or out.dtype != like.dtype or (
            not out.is_contiguous() if dense else out.shape[-1] > 1 and out.stride(-1) != 1):
        raise ValueError("out must be a %s tensor of shape %s and type %s on the inputs' GPU"
                         % ("contiguous" if dense else "(last axis contiguous)", tuple(like.shape), like.dtype))
    return out


def _rows(t):
    """`t` as rows of its last axis that one stride separates (copied where none does) and that stride."""
    n = t.shape[-1]
    if t.is_contiguous():
        return t, n
    flat = t.reshape(-1, n) if t.numel() else t.contiguous()
    return flat, (flat.stride(0) if flat.dim() == 2 and flat.shape[0] > 1 else n)


def _address(t):
    return None if t is None else t.data_ptr()


def _stream_handle(device):
    """The hipStream_t of the device's current stream.  A call of a few microseconds is made of such
    steps, so the handle is read without a stream object around it."""
    return _torch()._C._cuda_getCurrentRawStream(device.index)


def _workspace(workspace, need, device):
    """The scratch tensor (of the current stream, kept alive by the caller until the launch), its address
    and its bytes."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _torch().empty(need, dtype=_torch().uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if _scratch(workspace, device).numel() == 0:
        return None, None, 0
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _norm_params(X, scale, bias):
    cols, device = X.shape[-1], X.get_device()
    scale = _device_tensor(scale, "scale", device)
    for name, t in (("scale", scale), ("bias", bias)):
        if t is not None and tuple(t.shape) != (cols,):
            raise ValueError("%s must have shape (%d,)" % (name, cols))
    if scale.dtype != X.dtype and scale.dtype != _torch().float32:
        raise TypeError("scale must have X's element type or float32")
    if bias is not None:
        bias = _device_tensor(bias, "bias", device)
        if bias.dtype != scale.dtype:
            raise TypeError("bias must have scale's element type")
    return scale, bias


def layer_norm(X, scale, bias=None, epsilon: float = 1e-5, return_stats: bool = False, out=None,
               stream=None):
    """Layer normalisation over the last axis of X (gs_layer_norm).

    scale and bias have X's element type or float32.  With `return_stats` the
    mean and inverse standard deviation of each row are returned too (float32,
    X's shape without its last axis): layer_norm_backward takes them."""
    if stream is not None:
        return _on_stream(stream, layer_norm, X, scale, bias, epsilon, return_stats, out)
    torch = _torch()
    X = _tensor(X, "X")
    if X.dim() < 1:
        raise ValueError("X needs an axis")
    scale, bias = _norm_params(X, scale, bias)
    x, xs = _rows(X)
    cols = X.shape[-1]
    rows = X.numel() // cols if cols else math.prod(X.shape[:-1])
    Y = _output(out, X, True)
    mean = inv_std = None
    if return_stats:
        mean = torch.empty(X.shape[:-1], dtype=torch.float32, device=X.device)
        inv_std = torch.empty_like(mean)
    st = token_lib().gs_layer_norm(
        x.data_ptr(), dtype_code(X), rows, cols, xs, scale.data_ptr(), _address(bias), dtype_code(scale),
        epsilon, Y.data_ptr(), cols, _address(mean), _address(inv_std), _stream_handle(X.device))
    if st != GS_OK:
        _check(st, "gs_layer_norm")
    return (Y, mean, inv_std) if return_stats else Y


def layer_norm_backward(dY, X, scale, mean, inv_std, stream=None, workspace=None):
    """Gradients (dX, dscale, dbias) of layer_norm (gs_layer_norm_backward).
    `workspace`: device scratch; None takes it from torch's allocator."""
    if stream is not None:
        return _on_stream(stream, layer_norm_backward, dY, X, scale, mean, inv_std, workspace=workspace)
    torch = _torch()
    X = _tensor(X, "X")
    dY = _tensor(dY, "dY", X.get_device(), X.dtype, X.shape)
    scale, _ = _norm_params(X, scale, None)
    cols = X.shape[-1]
    rows = math.prod(X.shape[:-1])
    for name, t in (("mean", mean), ("inv_std", inv_std)):
        if t.dtype != torch.float32 or t.numel() != rows or t.get_device() != X.get_device():
            raise ValueError("%s must be a float32 tensor on X's GPU with an element per row" % name)
    mean, inv_std = mean.contiguous(), inv_std.contiguous()
    x, xs = _rows(X)
    dy, dys = _rows(dY)
    dX = _output(None, X, True)
    dscale, dbias = torch.empty_like(scale), torch.empty_like(scale)
    need = _I64(0)
    _check(token_lib().gs_layer_norm_backward_workspace_size(rows, cols, ctypes.byref(need)),
           "gs_layer_norm_backward_workspace_size")
    workspace, ws, ws_bytes = _workspace(workspace, need.value, X.device)
    st = token_lib().gs_layer_norm_backward(
        dy.data_ptr(), x.data_ptr(), dtype_code(X), rows, cols, dys, xs, scale.data_ptr(), dtype_code(scale),
        mean.data_ptr(), inv_std.data_ptr(), dX.data_ptr(), cols, dscale.data_ptr(), dbias.data_ptr(), ws,
        ws_bytes, _stream_handle(X.device))
    _check(st, "gs_layer_norm_backward")
    return dX, dscale, dbias


def dropout(X, ratio: float, seed: int, call: int = 0, residual=None, out=None, stream=None):
    """residual + dropout(X) (gs_dropout); the mask follows from seed, call and
    an element's place in X.  The gradient with respect to X is
    dropout(dY, ratio, seed, call); with respect to the residual it is dY."""
    if stream is not None:
        return _on_stream(stream, dropout, X, ratio, seed, call, residual, out)
    X = _device_tensor(X, "X")
    if residual is not None:
        residual = _device_tensor(residual, "residual", X.get_device())
        if residual.dtype != X.dtype or residual.shape != X.shape:
            raise ValueError("residual must have X's shape and element type")
    Y = _output(out, X, True)
    st = token_lib().gs_dropout(X.data_ptr(), dtype_code(X), X.numel(), _address(residual), ratio,
                                int(seed) & _MASK64, int(call) & _MASK32, Y.data_ptr(),
                                _stream_handle(X.device))
    if st != GS_OK:
        _check(st, "gs_dropout")
    return Y


def relative_bucket(r: int, num_buckets: int, max_distance: int = 128, bidirectional: int = 1) -> int:
    """Bucket of key position minus query position (gs_relative_bucket)."""
    got = _I(0)
    _check(token_lib().gs_relative_bucket(_whole(r, "r", *_INT64), _whole(num_buckets, "num_buckets"),
                                          _whole(max_distance, "max_distance"),
                                          _whole(bidirectional, "bidirectional"), ctypes.byref(got)),
           "gs_relative_bucket")
    return got.value


_INT64 = (-(2 ** 63), 2 ** 63 - 1)


def _whole(value, name, low=-(2 ** 31), high=2 ** 31 - 1):
    """`value` as a whole number that a field of the C interface holds (ctypes would cut it)."""
    value = int(value)
    if low <= value <= high:
        return value
    raise ValueError("%s must fit %d bits" % (name, high.bit_length() + 1))


def _strides(t):
    # the stride of an axis of one element addresses nothing
    (a, b, c, _), (i, j, k, _) = t.stride(), t.shape
    return a if i > 1 else 0, b if j > 1 else 0, c if k > 1 else 0


def _attention_inputs(Q, K, V, scale, causal, kv_lengths, table, max_distance, bidirectional,
                      q_position, ratio, seed, call):
    """Checked tensors of an attention call and its descriptor, without O's strides."""
    torch = _torch()
    if Q.dim() != 4 or K.dim() != 4:
        raise ValueError("Q and K must have shape (batch, heads, length, head_dim)")
    Q = _tensor(Q, "Q")
    device = Q.get_device()
    K = _tensor(K, "K", device, Q.dtype)
    if K.shape[0] != Q.shape[0] or K.shape[3] != Q.shape[3]:
        raise ValueError("K must share Q's batch and head_dim")
    V = _tensor(V, "V", device, Q.dtype, K.shape)
    B, H, Lq, D = Q.shape
    if kv_lengths is not None:
        kv_lengths = _tensor(kv_lengths, "kv_lengths", device, torch.int32, (B,)).contiguous()
    d = AttentionDesc()
    d.dtype = dtype_code(Q)
    d.batch, d.q_heads, d.q_len, d.head_dim = B, H, Lq, D
    d.kv_heads, d.kv_len = K.shape[1], K.shape[2]
    d.q_stride, d.k_stride, d.v_stride = _strides(Q), _strides(K), _strides(V)
    d.scale = 1.0 / math.sqrt(D) if scale is None and D else float(scale or 0.0)
    d.causal = _whole(causal, "causal")
    if isinstance(q_position, str):
        if q_position != "end":
            raise ValueError('q_position must be a number or "end"')
        d.q_from_end = 1
    else:
        d.q_position = _whole(q_position, "q_position", *_INT64)
    if table is not None:
        table = _device_tensor(table, "table", device)
        if table.dim() != 2 or table.shape[1] != H:
            raise ValueError("table must have shape (buckets, %d)" % H)
        if table.dtype != Q.dtype and table.dtype != torch.float32:
            raise TypeError("table must have Q's element type or float32")
        if table.shape[0] < 2:
            raise ValueError("table needs two buckets or more")
        d.table_dtype = dtype_code(table)
        d.num_buckets, d.max_distance = _whole(table.shape[0], "buckets"), _whole(max_distance, "max_distance")
        d.bidirectional = _whole(bidirectional, "bidirectional")
    else:
        d.table_dtype = GS_F32
    d.ratio, d.seed, d.call = ratio, int(seed) & _MASK64, int(call) & _MASK32
    return Q, K, V, kv_lengths, table, d


def attention(Q, K, V, scale=None, causal: int = 0, kv_lengths=None, table=None,
              max_distance: int = 128, bidirectional: int = 1, q_position=0, ratio: float = 0.0,
              seed: int = 0, call: int = 0, return_lse: bool = False, out=None, stream=None,
              workspace=None):
    """Attention with a relative position bias (gs_attention).

    Q (batch, heads, length, head_dim), K and V (batch, kv_heads, kv_length,
    head_dim), of any strides with a contiguous last axis: a (batch, length,
    heads, head_dim) tensor is passed as its transpose(1, 2).  `scale` defaults
    to 1 / sqrt(head_dim).  `kv_lengths` (int32, batch): keys each sequence
    holds.  `table` (buckets, heads): the learned bias.  `q_position`: position
    of query 0 among the keys, or "end" where the queries are the last of each
    sequence (a cache is read).  O is laid out like Q.  With `return_lse` the
    log-sum-exp of the scores (float32, batch x heads x length) is returned
    too: attention_backward takes it."""
    if stream is not None:
        return _on_stream(stream, attention, Q, K, V, scale, causal, kv_lengths, table, max_distance,
                          bidirectional, q_position, ratio, seed, call, return_lse, out, workspace=workspace)
    torch = _torch()
    Q, K, V, kv_lengths, table, d = _attention_inputs(
        Q, K, V, scale, causal, kv_lengths, table, max_distance, bidirectional, q_position, ratio,
        seed, call)
    O = _output(out, Q, False)
    d.o_stride = _strides(O)
    lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device) if return_lse else None
    if workspace is None:
        need = _I64(0)
        _check(token_lib().gs_attention_workspace_size(ctypes.byref(d), ctypes.byref(need)),
               "gs_attention_workspace_size")
        workspace, ws, ws_bytes = _workspace(None, need.value, Q.device)
    else:
        workspace, ws, ws_bytes = _workspace(workspace, 0, Q.device)
    st = token_lib().gs_attention(ctypes.byref(d), Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                  _address(kv_lengths), _address(table), O.data_ptr(), _address(lse), ws,
                                  ws_bytes, _stream_handle(Q.device))
    if st != GS_OK:
        _check(st, "gs_attention")
    return (O, lse) if return_lse else O


def attention_backward(dO, Q, K, V, O, lse, scale=None, causal: int = 0, kv_lengths=None, table=None,
                       max_distance: int = 128, bidirectional: int = 1, q_position=0,
                       ratio: float = 0.0, seed: int = 0, call: int = 0, stream=None,
                       workspace=None):
    """Gradients (dQ, dK, dV, dtable) of attention (gs_attention_backward) from
    its inputs, its O and its lse; dtable is None without a table."""
    if stream is not None:
        return _on_stream(stream, attention_backward, dO, Q, K, V, O, lse, scale, causal, kv_lengths, table,
                          max_distance, bidirectional, q_position, ratio, seed, call, workspace=workspace)
    torch = _torch()
    Q, K, V, kv_lengths, table, d = _attention_inputs(
        Q, K, V, scale, causal, kv_lengths, table, max_distance, bidirectional, q_position, ratio,
        seed, call)
    device = Q.get_device()
    O = _tensor(O, "O", device, Q.dtype, Q.shape)
    dO = _tensor(dO, "dO", device, Q.dtype, Q.shape)
    lse = _tensor(lse, "lse", device, torch.float32, Q.shape[:3]).contiguous()
    dQ, dK, dV = _like(Q), _like(K), _like(V)
    dtable = torch.empty_like(table) if table is not None else None
    d.o_stride, d.do_stride = _strides(O), _strides(dO)
    d.dq_stride, d.dk_stride, d.dv_stride = _strides(dQ), _strides(dK), _strides(dV)
    need = _I64(0)
    _check(token_lib().gs_attention_backward_workspace_size(ctypes.byref(d), ctypes.byref(need)),
           "gs_attention_backward_workspace_size")
    workspace, ws, ws_bytes = _workspace(workspace, need.value, Q.device)
    st = token_lib().gs_attention_backward(
        ctypes.byref(d), dO.data_ptr(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
        lse.data_ptr(), _address(kv_lengths), _address(table), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(),
        _address(dtable), ws, ws_bytes, _stream_handle(Q.device))
    _check(st, "gs_attention_backward")
    return dQ, dK, dV, dtable
