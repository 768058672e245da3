"""More small problems than one dispatch counts threads for (2^32): group norm of many small maps
and attention of many pairs of a batch element and a key head, against the definition in 64 bits."""

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
import norm_oracle
from attention_oracle import attention, check

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_of_many_small_maps(dtype):
    """32768 maps of 3 positions and 128 groups of one channel: 2^22 groups.  (The longest chain of
    additions is that of the parameters' gradients, 2048 maps: 8 sqrt(2100) u is within the oracle's
    2 ACC = 392 u.)"""
    kind = "f32" if dtype == torch.float32 else "bf16"
    B, P, C = 32768, 3, 128
    g = torch.Generator().manual_seed(11)
    x, go = (torch.randn((B, P, C), generator=g).to(dtype).cuda() for _ in range(2))
    w, b = (torch.randn(C, generator=g).to(dtype).cuda() for _ in range(2))
    out, mean, rstd = dcn.group_norm_act(x, C, w, b, activation="silu", return_stats=True)
    torch.cuda.synchronize()
    ref = norm_oracle.forward(f64(x), C, f64(w), f64(b), float(np.float32(1e-5)), "silu", kind)
    for n, t in (("mean", mean), ("rstd", rstd), ("out", out)):
        check(f64(t), ref[n], ref[n + "_tol"], n)
    del ref
    grads = dcn.group_norm_act_backward(go, x, mean, rstd, C, w, b, activation="silu")
    torch.cuda.synchronize()
    ref = norm_oracle.backward(f64(go), f64(x), f64(mean), f64(rstd), C, f64(w), f64(b), "silu", kind)
    for n, t in zip(("gx", "gw", "gb"), grads):
        check(f64(t), ref[n], ref[n + "_tol"], n)


def make_pairs(dtype):
    """One token of 16 heads of 8 on 8 key heads over 3 states, for 2^19 + 3 batch elements: more than
    2^22 pairs."""
    B, g = (1 << 19) + 3, torch.Generator().manual_seed(12)
    q, dout = (torch.randn((B, 1, 16, 8), generator=g).to(dtype).cuda() for _ in range(2))
    k, v = (torch.randn((B, 3, 8, 8), generator=g).to(dtype).cuda() for _ in range(2))
    mask = torch.rand((B, 3), generator=g).cuda() < 0.7
    return q, k, v, mask, dout


# the elements that are compared with 64 bits: the ends, and about those where a launch may end
SOME = [i + j for i in (0, 1 << 17, 1 << 18, 3 << 17, (1 << 19) - 1) for j in (0, 1, 2, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_of_many_small_pairs(dtype):
    q, k, v, mask, _ = make_pairs(dtype)
    out, lse = dcn.cross_attention(q, k, v, key_mask=mask, return_lse=True)
    torch.cuda.synchronize()
    ref = attention(*(f64(t[SOME]) for t in (q, k, v)), mask[SOME].cpu().numpy(), 8 ** -0.5,
                    "f32" if dtype == torch.float32 else "bf16")
    check(f64(out[SOME]), ref["out"], ref["out_tol"], "out")
    check(f64(lse[SOME]), ref["lse"], ref["lse_tol"], "lse")
    for at in range(0, q.shape[0], 1 << 17):     # every element, in calls of one launch
        piece = slice(at, at + (1 << 17))
        got = dcn.cross_attention(q[piece], k[piece], v[piece], key_mask=mask[piece], return_lse=True)
        assert torch.equal(got[0], out[piece]) and torch.equal(got[1], lse[piece]), at


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_gradients_of_many_small_pairs(dtype):
    """Over 2^24 workgroups of the gradients' launch: 2 for each of 2^23 pairs."""
    q, k, v, mask, dout = (torch.cat([t, t]) for t in make_pairs(dtype))
    out, lse = dcn.cross_attention(q, k, v, key_mask=mask, return_lse=True)
    grads = dcn.cross_attention_backward(dout, q, k, v, out, lse, key_mask=mask)
    torch.cuda.synchronize()
    last = [-1, -2, -3]
    ref = attention(*(f64(t[SOME + last]) for t in (q, k, v)), mask[SOME + last].cpu().numpy(), 8 ** -0.5,
                    "f32" if dtype == torch.float32 else "bf16", f64(dout[SOME + last]))
    for n, t in zip(("gq", "gk", "gv"), grads):
        check(f64(t[SOME + last]), ref[n], ref[n + "_tol"], n)
    for at in range(0, q.shape[0], 1 << 17):
        p = slice(at, at + (1 << 17))
        for x, y in zip(grads, dcn.cross_attention_backward(dout[p], q[p], k[p], v[p], out[p], lse[p], key_mask=mask[p])):
            assert torch.equal(x[p], y), at
