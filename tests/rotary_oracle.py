"""Rotary positions with several axes and their gradients in 64 bits on the CPU, written from the
definition pair by pair, and how far a result in fp32 or bf16 may be from them.

With u = 2^-24, e half a unit of bf16 (0 for fp32 data: its rounding is among the u) and acc(n) from
attention_oracle: a cosine or sine is off by 2^-23 and the angle's own error, 2^-51 of it; a turned element
is two products and a sum, 2 u (|x1| + |x2|) at most, and is rounded once."""

import numpy as np

from attention_oracle import E, U, acc

TINY = 1e-37   # results below fp32's smallest normal number may be flushed


def pairs_of(sections, layout):
    """(axis, first element, second element) of each pair."""
    total, out, start = sum(sections), [], 0
    for axis, n in enumerate(sections):
        for i in range(n):
            p = start + i
            out.append((axis,) + {"halves": (p, total + p), "adjacent": (2 * p, 2 * p + 1),
                                  "blocks": (2 * start + i, 2 * start + n + i)}[layout])
        start += n
    return out


def rotate(x, positions, frequencies, sections, layout, dtype, sign=1):
    """x [B,L,H,D], positions [B,L,axes], frequencies [pairs], float64 -> values and bounds."""
    y, tol = x.copy(), np.zeros_like(x)
    for p, (axis, i, j) in enumerate(pairs_of(sections, layout)):
        t = sign * positions[:, :, axis, None] * frequencies[p]
        c, s, a, b = np.cos(t), np.sin(t), x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        err = (2.0 ** -23 + 2.0 ** -51 * np.abs(t) + 2 * U) * (np.abs(a) + np.abs(b))
        tol[..., i] = err + E[dtype] * np.abs(y[..., i]) + TINY
        tol[..., j] = err + E[dtype] * np.abs(y[..., j]) + TINY
    return y, tol


def position_gradients(grad, x, positions, frequencies, sections, layout):
    """[B,L,axes]: the derivative of <rotate(x), grad> by each position, from d/dt (y1, y2) = (-y2, y1)."""
    out, tol = np.zeros(positions.shape), np.zeros(positions.shape)
    y, _ = rotate(x, positions, frequencies, sections, layout, "f32")
    n = x.shape[2] * sum(sections)
    for p, (axis, i, j) in enumerate(pairs_of(sections, layout)):
        f, t = frequencies[p], positions[:, :, axis, None] * frequencies[p]
        out[:, :, axis] += (f * (grad[..., j] * y[..., i] - grad[..., i] * y[..., j])).sum(2)
        # formed as gx2 x1 - gx1 x2 from the turned-back gradients
        size = np.abs(f) * (np.abs(grad[..., i]) + np.abs(grad[..., j])) * (np.abs(x[..., i]) + np.abs(x[..., j]))
        tol[:, :, axis] += ((2.0 ** -23 + 2.0 ** -51 * np.abs(t) + 6 * U + acc(n)) * size).sum(2)
    return out, tol + TINY
