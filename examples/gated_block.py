"""A block of the gated operators on a sampled feature map, trained, and read token by token.

    python examples/gated_block.py

Images are warped (affine_grid_sample_fused) and their positions read as tokens.
A gated recurrence mixes them along the sequence, residual_norm joins its
branch to the stream and normalises it for the gated feed-forward projections,
and a second residual_norm joins theirs.  Every gradient comes from the
operators' own backward calls.  The same block then runs a token at a time with
nothing but the recurrence's state kept; both give the same outputs.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spatial_transformer_grid_amd as gs  # noqa: E402

CHANNELS, HIDDEN = 48, 80


def parameters(width, dtype=torch.float32, device="cuda", seed=0):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, scale, mean=0.0):
        return (torch.randn(shape, generator=g, device=device) * scale + mean).to(dtype)

    p = {n: normal(width, scale=0.1, mean=1.0) for n in ("first", "post1", "pre2", "post2")}
    p.update({n: normal(width, scale=0.1, mean=0.5) for n in ("gate1", "gate2")})
    p.update(first_bias=normal(width, scale=0.1), mix=normal(width, 2 * CHANNELS, scale=width ** -0.5),
             out=normal(CHANNELS, width, scale=CHANNELS ** -0.5), gate=normal(HIDDEN, width, scale=width ** -0.5),
             up=normal(HIDDEN, width, scale=width ** -0.5), down=normal(HIDDEN, width, scale=HIDDEN ** -0.5))
    return p


def tokens(images, theta, spatial):
    """Warped images, a token a position: (batch, height * width, channels)."""
    warped = gs.affine_grid_sample_fused(theta, images, spatial, "linear", "zeros", 0)
    return warped.flatten(2).transpose(1, 2).contiguous()


def forward(x, p, lengths=None, state=None, last=None):
    """The block's output and what the backward pass needs; `state` and `last` as gated_recurrence takes them."""
    y, mean, inv_std = gs.layer_norm(x, p["first"], p["first_bias"], return_stats=True)
    values, gates = (y @ p["mix"]).split(CHANNELS, -1)  # strided views, as the operator takes them
    r, _, states = gs.gated_recurrence(values, gates, state, lengths, return_saved=True, last=last)
    b1 = r @ p["out"]
    h, z, stats1 = gs.residual_norm(x, b1, p["post1"], p["pre2"], gate=p["gate1"], return_stats=True)
    f, projections = gs.gated_linear(z, p["gate"], p["up"], return_saved=True)
    b2 = f @ p["down"]
    o, _, stats2 = gs.residual_norm(h, b2, p["post2"], gate=p["gate2"], return_stats=True)
    return o, (x, y, mean, inv_std, values, gates, r, states, b1, stats1, h, z, f, projections, b2, stats2)


def backward(do, saved, p, lengths=None):
    """Gradients of the parameters, and of x, from that of the block's output."""
    x, y, mean, inv_std, values, gates, r, states, b1, stats1, h, z, f, projections, b2, stats2 = saved
    flat = lambda t: t.flatten(0, 1)
    grads = {}
    dh, db2, grads["gate2"], grads["post2"], *_ = gs.residual_norm_backward(do, None, h, b2, stats2, p["post2"],
                                                                          gate=p["gate2"])
    grads["down"] = flat(f).t() @ flat(db2)
    dz, grads["gate"], grads["up"] = gs.gated_linear_backward(db2 @ p["down"].t(), z, p["gate"], p["up"], projections)
    dx, db1, grads["gate1"], grads["post1"], _, grads["pre2"], _ = gs.residual_norm_backward(
        dh, dz, x, b1, stats1, p["post1"], p["pre2"], gate=p["gate1"])
    grads["out"] = flat(r).t() @ flat(db1)
    dvalues, dgates, _ = gs.gated_recurrence_backward(db1 @ p["out"].t(), values, gates, states, lengths=lengths)
    dmix = torch.cat([dvalues, dgates], -1)
    grads["mix"] = flat(y).t() @ flat(dmix)
    dfirst, grads["first"], grads["first_bias"] = gs.layer_norm_backward(dmix @ p["mix"].t(), x, p["first"], mean, inv_std)
    return dx + dfirst, grads


def train(steps=30, rate=0.05, width=32, side=12):
    """Squared error to given tokens, plain gradient descent; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(1)
    images = torch.randn(4, width, side, side, generator=g, device="cuda")
    theta = torch.eye(2, 3, device="cuda").repeat(4, 1, 1) + 0.1 * torch.randn(4, 2, 3, generator=g, device="cuda")
    x, target = tokens(images, theta, (side, side)), torch.randn(4, side * side, width, generator=g, device="cuda") * 0.1
    p, losses = parameters(width), []
    for _ in range(steps):
        o, saved = forward(x, p)
        diff = o - x - target
        losses.append(float((diff * diff).mean()))
        _, grads = backward(2 * diff / diff.shape[0] / diff.shape[1], saved, p)
        for name, grad in grads.items():
            p[name] -= rate * grad
    return losses


def read_by_token(x, p):
    """The block over x, a token at a time, the recurrence's state kept in place."""
    state = torch.zeros(x.shape[0], CHANNELS, device=x.device)
    return torch.cat([forward(x[:, i:i + 1].contiguous(), p, state=state, last=state)[0] for i in range(x.shape[1])], 1)


def main():
    losses = train()
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
    x = torch.randn(2, 40, 32, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    p = parameters(32, seed=3)
    off = (read_by_token(x, p) - forward(x, p)[0]).abs().max()
    print("token by token against the whole sequence: largest difference %.2g" % off)


if __name__ == "__main__":
    main()
