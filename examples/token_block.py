"""A transformer block on a sampled feature map, trained, and read token by token.

    python examples/token_block.py

Images are warped (affine_grid_sample_fused), their positions read as tokens,
and a block of layer norm, attention with a learned relative position bias and
dropout with a residual is trained by hand-written steps: every gradient comes
from the operators' own backward calls.  The same block then runs causally
over a sequence and once more a token at a time from a cache of keys and
values; both give the same outputs.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spatial_transformer_grid_amd as gs  # noqa: E402

HEADS, KV_HEADS, DIM, BUCKETS, DISTANCE = 8, 4, 16, 16, 32


def parameters(width, dtype=torch.float32, device="cuda", seed=0):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, scale):
        return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)

    return {"scale": torch.ones(width, dtype=dtype, device=device),
            "bias": torch.zeros(width, dtype=dtype, device=device),
            "qkv": normal(width, (HEADS + 2 * KV_HEADS) * DIM, scale=width ** -0.5),
            "table": normal(BUCKETS, HEADS, scale=0.1),
            "out": normal(HEADS * DIM, width, scale=(HEADS * DIM) ** -0.5)}


def tokens(images, theta, spatial):
    """Warped images, a token a position: (batch, height * width, channels)."""
    warped = gs.affine_grid_sample_fused(theta, images, spatial, "linear", "zeros", 0)
    return warped.flatten(2).transpose(1, 2).contiguous()


def heads(y, p):
    """Queries, keys and values of normalised tokens, (batch, heads, tokens, DIM) without a copy."""
    qkv = (y @ p["qkv"]).unflatten(-1, (-1, DIM))
    return tuple(t.transpose(1, 2) for t in qkv.split([HEADS, KV_HEADS, KV_HEADS], 2))


def how(p, causal, seed, ratio, position=0):
    return dict(table=p["table"], max_distance=DISTANCE, causal=causal, bidirectional=1 - causal,
                q_position=position, ratio=ratio, seed=seed, call=0)


def forward(x, p, causal=0, seed=0, ratio=0.0):
    """x + dropout(attention(layer_norm(x))), and what the backward pass needs."""
    y, mean, inv_std = gs.layer_norm(x, p["scale"], p["bias"], return_stats=True)
    q, k, v = heads(y, p)
    o, lse = gs.attention(q, k, v, return_lse=True, **how(p, causal, seed, ratio))
    joined = o.transpose(1, 2).flatten(2)
    z = gs.dropout(joined @ p["out"], ratio, seed, call=1, residual=x)
    return z, (x, y, mean, inv_std, q, k, v, o, lse, joined)


def backward(dz, saved, p, causal=0, seed=0, ratio=0.0):
    """Gradients of the parameters, and of x, from that of the block's output."""
    x, y, mean, inv_std, q, k, v, o, lse, joined = saved
    d = gs.dropout(dz, ratio, seed, call=1)
    grads = {"out": joined.flatten(0, 1).t() @ d.flatten(0, 1)}
    do = (d @ p["out"].t()).unflatten(-1, (HEADS, DIM)).transpose(1, 2)
    dq, dk, dv, grads["table"] = gs.attention_backward(do, q, k, v, o, lse, **how(p, causal, seed, ratio))
    dqkv = torch.cat([t.transpose(1, 2) for t in (dq, dk, dv)], 2).flatten(2)
    grads["qkv"] = y.flatten(0, 1).t() @ dqkv.flatten(0, 1)
    dx, grads["scale"], grads["bias"] = gs.layer_norm_backward(dqkv @ p["qkv"].t(), x, p["scale"], mean, inv_std)
    return dx + dz, grads


def train(steps=30, rate=0.05, ratio=0.1, width=32, side=12):
    """Squared error to given tokens, plain gradient descent; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(1)
    images = torch.randn(4, width, side, side, generator=g, device="cuda")
    theta = torch.eye(2, 3, device="cuda").repeat(4, 1, 1) + 0.1 * torch.randn(4, 2, 3, generator=g, device="cuda")
    x, target = tokens(images, theta, (side, side)), torch.randn(4, side * side, width, generator=g, device="cuda") * 0.1
    p, losses = parameters(width), []
    for step in range(steps):
        z, saved = forward(x, p, seed=step, ratio=ratio)
        diff = z - x - target
        losses.append(float((diff * diff).mean()))
        _, grads = backward(2 * diff / diff.shape[0] / diff.shape[1], saved, p, seed=step, ratio=ratio)
        for name, grad in grads.items():
            p[name] -= rate * grad
    return losses


def read_by_token(x, p):
    """The causal block over x, a token at a time, the keys and values of earlier ones in a cache."""
    batch, length, _ = x.shape
    cache = torch.empty(2, batch, KV_HEADS, length, DIM, dtype=x.dtype, device=x.device)
    held = torch.zeros(batch, dtype=torch.int32, device=x.device)
    out = torch.empty_like(x)
    for i in range(length):
        token = x[:, i:i + 1].contiguous()
        q, k, v = heads(gs.layer_norm(token, p["scale"], p["bias"]), p)
        cache[0, :, :, i:i + 1], cache[1, :, :, i:i + 1] = k, v
        held += 1
        o = gs.attention(q, cache[0], cache[1], kv_lengths=held, **how(p, 1, 0, 0.0, "end"))
        out[:, i:i + 1] = token + o.transpose(1, 2).flatten(2) @ p["out"]
    return out


def main():
    losses = train()
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
    x = torch.randn(2, 40, 32, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    p = parameters(32, seed=3)
    off = (read_by_token(x, p) - forward(x, p, causal=1)[0]).abs().max()
    print("token by token against the whole sequence: largest difference %.2g" % off)


if __name__ == "__main__":
    main()
