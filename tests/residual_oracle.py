"""The join of two blocks (norms, gate, residual scale) and its gradients in 64 bits on the CPU, and
how far a result in fp32 or bf16 may be from them.

u, e and acc(n) as in attention_oracle.  An error is carried through each step by absolute values:
  - a row's mean is off by acc(C) of the mean of |f| and the mean of the errors of f;
  - the squares' sum is off by acc(C) of itself, and by twice the centred values' errors times them; the
    deviation's relative error is half that and a few u;
  - products and sums of a few terms add one u of their result each; outputs are rounded once."""

import numpy as np

from attention_oracle import E, U, acc

TINY = 1e-37


def norm(f, err, kind, eps):
    """The normed rows of f, known to +-err: values, bounds, mean, 1 / deviation, and bounds on those two."""
    one = np.ones_like(f[..., :1])
    if kind == "none":
        return f, err, 0 * one, one, 0 * one, 0 * one
    C = f.shape[-1]
    mean = f.mean(-1, keepdims=True) if kind == "layer" else 0 * one
    dmean = (acc(C) * np.abs(f).mean(-1, keepdims=True) + err.mean(-1, keepdims=True) + U * np.abs(mean)
             if kind == "layer" else 0 * one)
    d = f - mean
    derr = err + dmean + U * np.abs(d)
    var = (d * d).mean(-1, keepdims=True) + eps
    r = 1 / np.sqrt(var)
    drel = 0.5 * (acc(C) + 6 * U + (2 * np.abs(d) * derr + derr * derr).mean(-1, keepdims=True) / var) + 4 * U
    v = d * r
    return v, r * derr * (1 + drel) + np.abs(v) * (drel + U) + TINY, mean, r, dmean, r * drel


def affine(v, err, w, b):
    out = v if w is None else v * w
    err = err if w is None else np.abs(w) * err + U * np.abs(out)
    if b is not None:
        out = out + b
        err = err + U * np.abs(out)
    return out, err


def wide(t, like):
    """A gate [B,C] or [B,P,C], or a vector [C], over rows [B,P,C]."""
    return t if t.ndim != 2 else t[:, None] + 0 * like


def forward(x, y, gate, scale, n1, w1, b1, n2, w2, b2, eps, dtype):
    """x, y [B,P,C] float64 -> dict of values and bounds."""
    e = E[dtype]
    v, verr, m1, r1, dm1, dr1 = norm(y, np.zeros_like(y), n1, eps)
    z, zerr = affine(v, verr, w1, b1)
    f = np.ones_like(x)
    if gate is not None:
        f = f * wide(gate, x)
    if scale is not None:
        f = f * scale
    o = x + f * z
    oerr = np.abs(f) * zerr + 2 * U * np.abs(f * z) + U * np.abs(o)
    u, uerr, m2, r2, dm2, dr2 = norm(o, oerr, n2, eps)
    nxt, nerr = affine(u, uerr, w2, b2)
    return {"out": o, "out_tol": oerr + e * np.abs(o) + TINY, "next": nxt, "next_tol": nerr + (e + U) * np.abs(nxt) + TINY,
            "stats": np.concatenate((m1, r1, m2, r2), -1),
            "stats_tol": np.concatenate((dm1, dr1, dm2, dr2), -1) * 1.01 + TINY}


def norm_gradient(g, gerr, v, verr, r, kind):
    """r (g - mean(g) - v mean(g v)), and its bound."""
    if kind == "none":
        return g, gerr
    C = g.shape[-1]
    mg = g.mean(-1, keepdims=True) if kind == "layer" else 0 * g[..., :1]
    mv = (g * v).mean(-1, keepdims=True)
    dmg = acc(C + 1) * np.abs(g).mean(-1, keepdims=True) + gerr.mean(-1, keepdims=True) if kind == "layer" else 0 * mg
    dmv = acc(C + 1) * np.abs(g * v).mean(-1, keepdims=True) + (np.abs(g) * verr + np.abs(v) * gerr).mean(-1, keepdims=True)
    size = np.abs(g) + np.abs(mg) + np.abs(v * mv)
    return r * (g - mg - v * mv), r * (gerr + dmg + np.abs(v) * dmv + verr * np.abs(mv) + 5 * U * size)


def backward(go, gn, x, y, stats, gate, scale, n1, w1, b1, n2, w2, dtype):
    """Gradients from the statistics that the call is given -> dict of values and bounds."""
    e, C = E[dtype], x.shape[-1]
    rows = x.shape[0] * x.shape[1]
    m1, r1, m2, r2 = (stats[..., i:i + 1] for i in range(4))
    v = (y - m1) * r1
    verr = 3 * U * np.abs(v) + U * np.abs(y * r1) if n1 != "none" else 0 * v
    z, zerr = affine(v, verr, w1, b1)
    g = wide(gate, x) if gate is not None else np.ones_like(x)
    s = np.ones(C) if scale is None else scale
    f = g * s
    d = np.zeros_like(x) if go is None else go.copy()
    derr = np.zeros_like(x)
    sums = {}
    if n2 != "none":
        o = x + f * z
        oerr = np.abs(f) * zerr + 2 * U * np.abs(f * z) + U * np.abs(o)
        u = (o - m2) * r2
        uerr = r2 * (oerr + U * np.abs(o - m2)) + 2 * U * np.abs(u)
        gn = np.zeros_like(x) if gn is None else gn
        sums["gw2"], sums["gb2"] = (gn * u, np.abs(gn) * uerr), (gn, 0 * gn)
        gu = gn if w2 is None else gn * w2
        t, terr = norm_gradient(gu, U * np.abs(gu), u, uerr, r2, n2)
        d = d + t
        derr = terr + U * (np.abs(d) + np.abs(t))
    res = {"gx": d, "gx_tol": derr + (e + U) * np.abs(d) + TINY}
    dz, dzerr = d * z, derr * np.abs(z) + np.abs(d) * zerr + 2 * U * np.abs(d * z)
    if gate is not None:
        gg, ggerr = dz * s, np.abs(s) * dzerr + 2 * U * np.abs(dz * s)
        if gate.ndim == 2:
            n = x.shape[1]
            res["ggate"] = gg.sum(1)
            res["ggate_tol"] = (ggerr + acc(n) * np.abs(gg)).sum(1) + (e + 2 * U) * np.abs(res["ggate"]) + TINY
        else:
            res["ggate"], res["ggate_tol"] = gg, ggerr + (e + U) * np.abs(gg) + TINY
    sums["gscale"] = (dz * g, np.abs(g) * dzerr + 2 * U * np.abs(dz * g))
    h = d * f
    herr = np.abs(f) * derr + 3 * U * np.abs(h)
    sums["gw1"], sums["gb1"] = (h * v, np.abs(v) * herr + np.abs(h) * verr + 2 * U * np.abs(h * v)), (h, herr)
    gv = h if w1 is None else h * w1
    gverr = herr if w1 is None else np.abs(w1) * herr + U * np.abs(gv)
    gy, gyerr = norm_gradient(gv, gverr, v, verr, r1, n1)
    res["gy"], res["gy_tol"] = gy, gyerr + (e + U) * np.abs(gy) + TINY
    for n, (term, err) in sums.items():
        res[n] = term.sum((0, 1))
        res[n + "_tol"] = (err + acc(rows) * np.abs(term)).sum((0, 1)) + (e + 3 * U) * np.abs(res[n]) + TINY
    return res
