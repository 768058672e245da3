"""Channels-last group normalisation with an activation, and its gradients, in 64 bits on the
CPU, written from the definition, and how far a result in fp32 or bf16 may be from them.

The bounds follow the arithmetic that include/dcn.h states (u, e: half units of fp32 and bf16,
as in attention_oracle).  A sum whose longest chain of additions is h long is off by at most
8 sqrt(h) u times the sum of absolute values; at the tests' sizes no chain is longer than
CHAIN.  Squares are summed about a value of the channel, so the variance's error goes by
var + (the largest deviation)^2, and not by the mean's square."""

import numpy as np
from scipy.special import erf

from attention_oracle import E, U

CHAIN = 600
ACC = 8.0 * np.sqrt(CHAIN) * U


def activate(z, act):
    if act == "relu":
        return np.maximum(z, 0)
    if act == "silu":
        return z / (1 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + erf(z / np.sqrt(2)))
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + erf(z / np.sqrt(2))) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    return np.ones_like(z)


# the largest slopes of the activations and of their slopes
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13}
BEND = {"none": 0.0, "relu": 0.0, "silu": 0.5, "gelu": 0.8}


def _groups(t, G):
    b, c = t.shape[0], t.shape[-1]
    return t.reshape(b, -1, G, c // G)


def _param(t, G, C, default):
    t = np.full(C, default) if t is None else t
    return t.reshape(1, 1, G, C // G)


def forward(x, G, weight, bias, eps, act, dtype):
    C = x.shape[-1]
    xg, w, b = _groups(x, G), _param(weight, G, C, 1.0), _param(bias, G, C, 0.0)
    mean = xg.mean((1, 3), keepdims=True)
    dev = xg - mean
    var = (dev ** 2).mean((1, 3), keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    most = np.abs(dev).max((1, 3), keepdims=True)
    n = dev * rstd
    z = n * w + b
    y = activate(z, act)
    # deviations are taken from a value of the channel: at most twice the largest one
    mean_tol = 2 * ACC * most + 4 * U * np.abs(mean) + 1e-37
    var_tol = 2 * ACC * (var + 4 * most ** 2) + mean_tol ** 2
    rstd_tol = rstd * (0.5 * var_tol / (var + eps) + 8 * U)
    z_tol = np.abs(w) * (rstd * mean_tol + np.abs(dev) * rstd_tol) + 6 * U * (np.abs(n * w) + np.abs(b))
    y_tol = LIPSCHITZ[act] * z_tol + 4 * U * (np.abs(z) + 8) * np.abs(z) + (E[dtype] + U) * np.abs(y) + 1e-37
    return {"out": y.reshape(x.shape), "out_tol": y_tol.reshape(x.shape), "mean": mean[:, 0, :, 0],
            "mean_tol": mean_tol[:, 0, :, 0], "rstd": rstd[:, 0, :, 0], "rstd_tol": rstd_tol[:, 0, :, 0]}


def backward(g, x, mean, rstd, G, weight, bias, act, dtype):
    """mean and rstd [B,G]: the statistics the call is given."""
    C, e = x.shape[-1], E[dtype]
    xg, gg = _groups(x, G), _groups(g, G)
    w, b = _param(weight, G, C, 1.0), _param(bias, G, C, 0.0)
    mean, rstd = mean[:, None, :, None], rstd[:, None, :, None]
    N = xg.shape[1] * xg.shape[3]
    n = (xg - mean) * rstd
    z = n * w + b
    n_err = 3 * U * np.abs(n)
    z_err = 6 * U * (np.abs(n * w) + np.abs(b))
    s = slope(z, act)
    s_err = BEND[act] * z_err + (16 * U * (1 + np.abs(z)) ** 2 if act in ("silu", "gelu") else 0)
    if act == "relu":                       # the slope jumps at 0: either side within the argument's error
        s_err = (np.abs(z) <= z_err).astype(np.float64)
    gz = gg * s
    gz_err = np.abs(gg) * s_err + 2 * U * np.abs(gz)
    gn_err = gz_err * np.abs(n) + np.abs(gz) * n_err + 2 * U * np.abs(gz * n)
    r = {}
    for name, v, err in (("gw", gz * n, gn_err), ("gb", gz, gz_err)):
        t = v.sum((0, 1)).reshape(C)
        r[name] = t
        r[name + "_tol"] = (err.sum((0, 1)) + 2 * ACC * np.abs(v).sum((0, 1))).reshape(C) + (e + U) * np.abs(t) + 1e-37
    m1, m2 = ((w * t).sum((1, 3), keepdims=True) / N for t in (gz, gz * n))
    m1_err, m2_err = ((np.abs(w) * err + 2 * ACC * np.abs(w * t)).sum((1, 3), keepdims=True) / N + 2 * U * np.abs(m)
                      for t, err, m in ((gz, gz_err, m1), (gz * n, gn_err, m2)))
    gx = rstd * (w * gz - m1 - n * m2)
    gx_err = rstd * (np.abs(w) * gz_err + m1_err + np.abs(n) * m2_err + n_err * np.abs(m2) +
                     6 * U * (np.abs(w * gz) + np.abs(m1) + np.abs(n * m2))) + (e + U) * np.abs(gx) + 1e-37
    r["gx"], r["gx_tol"] = gx.reshape(x.shape), gx_err.reshape(x.shape)
    return r
