"""Cross attention and its gradients where keys are many: the windows of mask bits are read again
(over 2048 keys in the rows form and the gradients, over 64 turns of the few-rows form), rings of
tiles go round, keys are split over many workgroups, rows are read element by element.  Keys and
values are shared by the batch (stride 0), each batch element has a mask of another kind, and some
pairs of a batch element and a key head are compared with the definition in 64 bits within the
bounds of attention_oracle.  The workspace shows that a case is split as it is meant to be."""

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
from attention_oracle import E, U, check, one_head

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPES = [("f32", 32), ("f32", 64), ("f32", 128), ("f32", 37), ("f32", 125), ("bf16", 32), ("bf16", 64), ("bf16", 128),
         ("bf16", 20), ("bf16", 60), ("bf16", 100)]


def padded(D):
    return 32 if D <= 32 else 64 if D <= 64 else 128


def turn(dtype, D):
    """Keys of one turn of a few-rows workgroup: 32 of each wave."""
    return 32 * ({32: 16, 64: 8, 128: 8} if dtype == "bf16" else {32: 16, 64: 8, 128: 4})[padded(D)]


def masks(B, Lk, g):
    """Row i: all kept; islands of a few keys between long gaps; the last 30 keys only; six in ten; none;
    a run that ends inside a tile."""
    m = torch.zeros((B, Lk), dtype=torch.bool)
    for i in range(B):
        if i % 6 == 0:
            m[i] = True
        elif i % 6 == 1:
            for at in range(700, Lk, 2300):
                m[i, at:at + 3] = True
        elif i % 6 == 2:
            m[i, -30:] = True
        elif i % 6 == 3:
            m[i] = torch.rand(Lk, generator=g) < 0.6
        elif i % 6 == 5:
            m[i, :Lk - 71] = True
    return m


def make(dtype, B, Lq, Lk, Hq, Hkv, D):
    g = torch.Generator().manual_seed(1000 * D + Lk + B)
    t = DT[dtype]
    q, dout = (torch.randn((B, Lq, Hq, D), generator=g).to(t).cuda() for _ in range(2))
    k, v = (torch.randn((1, Lk, Hkv, D), generator=g).to(t).cuda().expand(B, Lk, Hkv, D) for _ in range(2))
    return q, k, v, masks(B, Lk, g).cuda(), dout


def f64(t):
    return t.double().cpu().numpy()


def compare(dtype, q, k, v, m, dout, pairs, what):
    print(f"[gpu-test] attention {what} {dtype} {tuple(q.shape)} over {tuple(k.shape)}", flush=True)
    (B, Lq, Hq, D), Hkv = q.shape, k.shape[2]
    g, scale = Hq // Hkv, D ** -0.5
    out, lse = dcn.cross_attention(q, k, v, key_mask=m, return_lse=True)
    grads = dcn.cross_attention_backward(dout, q, k, v, out, lse, key_mask=m)
    torch.cuda.synchronize()
    assert torch.equal(dcn.cross_attention(q, k, v, key_mask=m), out), "the same call gave other bits"
    keep = m.cpu().numpy()
    for b, hk in pairs:
        heads = slice(hk * g, (hk + 1) * g)
        at = np.flatnonzero(keep[b])
        kk, vv = f64(k[0, :, hk])[at], f64(v[0, :, hk])[at]
        qq, dd, oo, ll, gq = (f64(t) for t in (q[b, :, heads], dout[b, :, heads], out[b, :, heads], lse[b, heads],
                                               grads[0][b, :, heads]))
        sums = {n: 0.0 for n in ("gk", "gk_tol", "gv", "gv_tol")}
        for h in range(g):
            r = one_head(qq[:, h], kk, vv, scale, dtype, dd[:, h])
            where = f"element {b} key head {hk} head {h} "
            check(oo[:, h], r["out"], r["out_tol"], where + "out")
            check(ll[h], r["lse"], r["lse_tol"], where + "lse")
            check(gq[:, h], r["gq"], r["gq_tol"], where + "gq")
            for n in sums:
                sums[n] = sums[n] + r[n]
        for n, t in (("gk", grads[1]), ("gv", grads[2])):
            want, tol = (np.zeros((k.shape[1], D)) for _ in range(2))
            want[at] = sums[n]
            tol[at] = sums[n + "_tol"] + (E[dtype] + (4 + g) * U) * np.abs(sums[n]) + 1e-37
            check(f64(t[b, :, hk]), want, tol, f"element {b} key head {hk} {n}")


def splits(q, k, v, m, rows):
    """Parts of a tile of the forward, where all of them are split alike; 1: no tile is split."""
    B, Lq, Hq, D = q.shape
    tiles = B * k.shape[2] * -(-Lq * (Hq // k.shape[2]) // rows)
    nbytes = dcn.dcn_cross_attention_workspace_bytes(dcn.attention_desc(q, k, v, m))
    return max(1, nbytes // (tiles * rows * (padded(D) * 4 + 8)))


@pytest.mark.parametrize("dtype,D", TYPES)
def test_few_rows_over_more_than_a_window_of_keys(dtype, D):
    """256 tiles of one token: unsplit, more than 64 turns of each workgroup."""
    x = make(dtype, 16, 1, 65 * turn(dtype, D) + 77, 32, 16, D)
    assert splits(*x[:4], 32) == 1
    compare(dtype, *x, [(0, 0), (1, 3), (2, 15), (3, 7), (4, 1), (5, 12), (15, 15)], "one token, windows")


@pytest.mark.parametrize("dtype,D", TYPES)
def test_few_rows_in_many_parts(dtype, D):
    x = make(dtype, 6, 2, 17003, 3, 1, D)
    assert splits(*x[:4], 32) >= 7
    compare(dtype, *x, [(b, 0) for b in range(6)], "two tokens in parts")


@pytest.mark.parametrize("dtype,D", [("f32", 128), ("f32", 125), ("bf16", 128), ("bf16", 100)])
def test_few_rows_in_two_parts_of_more_than_a_window(dtype, D):
    x = make(dtype, 8, 1, 2 * 64 * turn(dtype, D) + 600, 16, 16, D)
    assert splits(*x[:4], 32) == 2
    compare(dtype, *x, [(0, 0), (1, 3), (2, 15), (3, 7), (5, 12)], "one token, windows in parts")


@pytest.mark.parametrize("B,dtype,D", [(8, *x) for x in TYPES] + [(12, "bf16", 32), (12, "bf16", 20)])
def test_rows_over_more_than_a_window_of_keys(B, dtype, D):
    """512 tiles of 128 rows, unsplit, over 71 tiles of keys.  The gradients' rounds of the chip are
    256, 512 or 768 tiles: at bf16 heads of 32 it takes 768 for theirs to be unsplit."""
    x = make(dtype, B, 512, 4500, 16, 16, D)
    if B == 8:
        assert splits(*x[:4], 128) == 1
    if B == 12 or (dtype, padded(D)) != ("bf16", 32):
        assert dcn.dcn_cross_attention_backward_workspace_bytes(dcn.attention_desc(*x[:4])) == B * 16 * 512 * 8
    compare(dtype, *x, [(0, 0), (1, 9), (2, 15), (3, 4)], "rows, windows")


@pytest.mark.parametrize("dtype,D", TYPES)
def test_rows_in_many_parts(dtype, D):
    x = make(dtype, 6, 250, 4500, 6, 3, D)
    assert splits(*x[:4], 128) == 7
    compare(dtype, *x, [(b, b % 3) for b in range(6)], "rows in parts")
