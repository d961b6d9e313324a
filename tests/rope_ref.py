"""Plain fp64 forms of the head norm and rotation and of their backward, from
their definitions, for the tests of the CUDA path."""

from __future__ import annotations

import torch


def frequencies(dim, base):
    i = torch.arange(dim // 2, dtype=torch.float64)
    return base ** (-2.0 * i / dim)


def angles(positions, freq, axes):
    """[B, S, dim / 2] from positions [axes, B, S]."""
    return torch.stack([positions[a].double() * f
                        for a, f in zip(axes, freq.tolist())], -1)


def turn(x, angle, interleaved, sign=1.0):
    """Rows x [B, h, S, D] (fp64) with their first pairs turned by sign *
    angle [B, S, dim / 2]."""
    half = angle.shape[-1]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None] * sign
    y = x.clone()
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def sizes(x, half, interleaved):
    """Per element the length of its pair (its own magnitude where it does not
    turn): what an absolute error of a cosine is multiplied with."""
    y = x.abs().clone()
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    y[..., a] = y[..., b] = torch.hypot(x[..., a], x[..., b])
    return y


def forward(x, w, eps, angle, interleaved):
    """(result, size) in fp64; w, eps, angle None where there is none."""
    x = x.double()
    if eps is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        x = x if w is None else x * w.double()
    if angle is None:
        return x, x.abs()
    return (turn(x, angle, interleaved),
            sizes(x, angle.shape[-1], interleaved))


def backward(g, x, w, eps, angle, interleaved):
    """(dx, its size, dw, its size) in fp64."""
    h = g.double()
    hs = h.abs()
    if angle is not None:
        hs = sizes(h, angle.shape[-1], interleaved)
        h = turn(h, angle, interleaved, -1.0)
    if eps is None:
        return h, hs, None, None
    r = 1.0 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + eps)
    n = x.double() * r
    one = torch.ones(x.shape[-1], dtype=torch.float64)
    w = one if w is None else w.double()
    m = (h * w * n).mean(-1, keepdim=True)
    ms = (hs * w.abs() * n.abs()).mean(-1, keepdim=True)
    dx = r * (h * w - n * m)
    return (dx, r * (hs * w.abs() + n.abs() * ms), (h * n).sum((0, 1, 2)),
            (hs * n.abs()).sum((0, 1, 2)))
