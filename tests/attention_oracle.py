"""Cross attention and its gradients in 64 bits on the CPU, written from the definition, and
how far a result in fp32 or bf16 may be from them.

The bounds follow the arithmetic that include/dcn.h states.  With u = 2^-24 (half a unit of
fp32) and e = 2^-9 (half a unit of bf16; 0 for fp32 data):
  - a sum of n products or terms in fp32, in any order, is off by at most
    8 sqrt(n + 1) u times the sum of their absolute values (rounding errors as independent
    variables of mean 0: the chance of more is below exp(-32));
  - the scores' error enters the weights through exp: a weight's relative error is the score's
    absolute error, twice (its own and its row sum's), and 16 u for the exponential's argument
    and value;
  - each rounding to bf16 that dcn.h names adds e times the absolute value of what it rounds,
    carried through the sums by absolute values."""

import numpy as np
import torch

# half of the format's spacing at 1
U = torch.finfo(torch.float32).eps / 2
E = {"f32": 0.0, "bf16": torch.finfo(torch.bfloat16).eps / 2}


def acc(n):
    return 8.0 * np.sqrt(n + 1.0) * U


def one_head(q, k, v, scale, dtype, dout=None, out_rounded=None):
    """One batch element and head over its attended keys: q [Lq,D], k and v [n,D] float64.
    Returns a dict of values and of bounds on the error of each."""
    lq, d = q.shape
    n, e = k.shape[0], E[dtype]
    r = {}
    if n == 0:
        z = np.zeros((lq, d))
        r.update(out=z, out_tol=z, lse=np.full(lq, -np.inf), lse_tol=np.zeros(lq), gq=z, gq_tol=z,
                 gk=np.zeros((0, d)), gk_tol=np.zeros((0, d)), gv=np.zeros((0, d)), gv_tol=np.zeros((0, d)))
        return r
    s = scale * (q @ k.T)
    s_abs = scale * (np.abs(q) @ np.abs(k).T)
    ds = (acc(d) + 4 * U) * s_abs + 4 * U * np.abs(s).max(1, keepdims=True)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    total = w.sum(1, keepdims=True)
    p = w / total
    lse = (m + np.log(total))[:, 0]
    dw = 2 * ds.max(1, keepdims=True) + acc(n) + 16 * U          # relative error of a weight
    out = p @ v
    va = p @ np.abs(v)
    # 1e-37: results below fp32's smallest normal number may be flushed
    r.update(out=out, out_tol=(dw + acc(n) + 1.01 * e) * va + (e + U) * np.abs(out) + 1e-37, lse=lse,
             lse_tol=dw[:, 0] + 4 * U * np.abs(lse) + 4 * U)
    if dout is None:
        return r
    dp = dout @ v.T
    delta = (dout * out).sum(1, keepdims=True)
    dsc = p * (dp - delta)
    err_dp = acc(d) * (np.abs(dout) @ np.abs(v).T)
    # delta is formed from the rounded output
    err_delta = acc(d) * (np.abs(dout) * np.abs(out)).sum(1, keepdims=True) + \
        (np.abs(dout) * r["out_tol"]).sum(1, keepdims=True)
    dwb = dw + 4 * U * np.abs(lse)[:, None]
    err_ds = dwb * np.abs(dsc) + p * (err_dp + err_delta) * (1 + dwb) + 4 * U * np.abs(dsc) + 1.01 * e * np.abs(dsc)
    gq, gk, gv = scale * (dsc @ k), scale * (dsc.T @ q), p.T @ dout
    r.update(gq=gq, gk=gk, gv=gv)
    r["gq_tol"] = scale * ((err_ds + acc(n) * np.abs(dsc)) @ np.abs(k)) + (e + 4 * U) * np.abs(gq) + 1e-37
    # dK and dV add up rows (and heads): the caller adds their bounds; their rounding comes last
    r["gk_tol"] = scale * ((err_ds + acc(lq) * np.abs(dsc)).T @ np.abs(q))
    r["gv_tol"] = ((dwb + acc(lq) + 1.01 * e) * p).T @ np.abs(dout)
    return r


def attention(q, k, v, mask, scale, dtype, dout=None):
    """[B,L,H,D] float64 arrays (mask [B,Lk] bool or None) -> dict of arrays and bounds."""
    b, lq, hq, d = q.shape
    lk, hkv = k.shape[1], k.shape[2]
    g = hq // hkv
    names = ["out", "out_tol"] + (["gq", "gq_tol"] if dout is not None else [])
    res = {n: np.zeros((b, lq, hq, d)) for n in names}
    res["lse"], res["lse_tol"] = np.zeros((b, hq, lq)), np.zeros((b, hq, lq))
    if dout is not None:
        for n in ("gk", "gk_tol", "gv", "gv_tol"):
            res[n] = np.zeros((b, lk, hkv, d))
    for i in range(b):
        at = np.arange(lk) if mask is None else np.flatnonzero(mask[i])
        for h in range(hq):
            r = one_head(q[i, :, h], k[i, at, h // g], v[i, at, h // g], scale, dtype,
                         None if dout is None else dout[i, :, h])
            for n in names:
                res[n][i, :, h] = r[n]
            res["lse"][i, h], res["lse_tol"][i, h] = r["lse"], r["lse_tol"]
            if dout is not None:
                for n in ("gk", "gk_tol", "gv", "gv_tol"):
                    res[n][i, at, h // g] += r[n]
    if dout is not None:
        for n in ("gk", "gv"):
            kept = np.ones((b, lk), bool) if mask is None else mask
            res[n + "_tol"] += ((E[dtype] + (4 + g) * U) * np.abs(res[n]) + 1e-37) * kept[:, :, None, None]
    return res


def check(got, want, tol, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, f"{what}: shape {got.shape}, not {want.shape}"
    same = got == want                     # infinities of one sign too
    with np.errstate(invalid="ignore"):
        off = np.where(same, 0.0, np.abs(got - want))
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} values outside their bound, the worst " \
        f"{np.nanmax(np.where(bad, off / np.maximum(tol, 1e-300), 0)):.2f} times it; {int(np.isnan(got).sum())} NaN; " \
        f"first at {tuple(np.argwhere(bad)[0])}: {got[bad][0]!r} for {want[bad][0]!r}"
