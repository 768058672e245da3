"""dcn_paged_attention holds its softmax weights in fp32 for bf16 data too: against the definition in 64
bits, within the fp32 bounds of attention_oracle and one rounding of the output.

For bf16 a weight is three products of 8 bits, exactly, so an output is a sum of 3n products in fp32 in
place of n: acc(3n) for acc(n)."""

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
from attention_oracle import E, acc, check, one_head
from test_gpu_paged import ATTENTION, DT, f64, make, tables

pytestmark = pytest.mark.gpu


def reference(q, k, v, table, lengths, dtype, scale):
    """out, lse and their bounds, with weights of fp32 whatever the data's type."""
    q, k, v, table, lengths = f64(q), f64(k), f64(v), table.cpu().numpy(), lengths.cpu().numpy()
    B, hq, d = q.shape
    page, hkv = k.shape[1:3]
    g = hq // hkv
    out, tol, lse, ltol = np.zeros_like(q), np.zeros_like(q), np.zeros((B, hq)), np.zeros((B, hq))
    for b in range(B):
        j = np.arange(lengths[b])
        at, place = table[b][j // page], j % page
        n = len(j)
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            keys, values = k[at, place, h], v[at, place, h]
            r = one_head(q[b, rows], keys, values, scale, "f32")
            out[b, rows], lse[b, rows], ltol[b, rows] = r["out"], r["lse"], r["lse_tol"]
            tol[b, rows] = r["out_tol"] + E[dtype] * np.abs(r["out"])
            if dtype == "bf16":
                tol[b, rows] += (acc(3 * n) - acc(n)) * one_head(q[b, rows], keys, np.abs(values), scale, "f32")["out"]
    return out, tol, lse, ltol


def compare(args, dtype, what, scale):
    out, lse = dcn.paged_attention(*args, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    want, tol, wl, tl = reference(*args, dtype, scale)
    check(f64(out), want, tol, what + " out")
    check(f64(lse), wl, tl, what + " lse")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128, 8, 37])
def test_outputs_that_nearly_cancel(dtype, d):
    """Three positions: one of weight 1 and value 0, and two of weights about 0.51 whose values are each other's
    negatives, so that an output is the difference of two weights and its own rounding tells nothing away."""
    print(f"[gpu-test] paged weights {dtype} {d}", flush=True)
    g = torch.Generator().manual_seed(d)
    B, hq, hkv, page, t = 33, 8, 2, 4, DT[dtype]
    table = tables([1] * B, B, 1, g)
    q, k, v = torch.zeros(B, hq, d), torch.zeros(B, page, hkv, d), torch.zeros(B, page, hkv, d)
    q[:, :, 0] = 0.97 + 0.06 * torch.rand((B, hq), generator=g)
    k[:, 1, :, 0] = -0.68 + 0.01 * torch.rand((B, hkv), generator=g)
    k[:, 2, :, 0] = k[:, 1, :, 0] + 0.004
    v[:, 1] = torch.randn((B, hkv, d), generator=g)
    v[:, 2] = -v[:, 1]
    lengths = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    compare([a.to(t).cuda() for a in (q, k, v)] + [table, lengths], dtype, f"d {d}", 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(ATTENTION))
def test_values_of_alternating_signs(name, dtype):
    """The sequences of test_gpu_paged, with small scores and values that alternate from position to position."""
    print(f"[gpu-test] paged weights {name} {dtype}", flush=True)
    q, k, v, table, lengths = make(name, dtype, seed=1, scale=0.02)
    page = k.shape[1]
    sign = torch.ones(v.shape[:2], device="cuda")
    for b, n in enumerate(lengths.tolist()):
        j = torch.arange(n, device="cuda")[1::2]
        sign[table[b].long()[j // page], j % page] = -1
    v = (v.float().abs() * sign[:, :, None, None]).to(v.dtype)
    compare((q, k, v, table, lengths), dtype, name, q.shape[2] ** -0.5)


def test_infinite_values_under_any_weight():
    """A weight's three operands are positive wherever the weight is: no infinite value becomes NaN."""
    g = torch.Generator().manual_seed(7)
    B, page, d = 257, 4, 32
    table = tables([1] * B, B, 1, g)
    q, k, v = torch.zeros(B, 2, d), torch.zeros(B, page, 2, d), torch.randn((B, page, 2, d), generator=g)
    q[:, :, 0] = 1
    # weights from 1 down to 2^-90, powers of two (no bits but the first) among them
    k[:, 1, :, 0] = -torch.linspace(0, 90, B)[:, None] * float(np.log(2))
    k[::3, 1, :, 0] = 0
    v[:, 1, :, ::2] = float("inf")
    lengths = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    out = dcn.paged_attention(*(a.bfloat16().cuda() for a in (q, k, v)), table, lengths, scale=1.0)
    assert torch.all(out[..., ::2] == float("inf")) and torch.isfinite(out[..., 1::2]).all()


def test_infinite_values_under_the_least_weights():
    """Down to fp32's least normal number, below which a weight may be 0."""
    g = torch.Generator().manual_seed(8)
    B, page, d = 260, 4, 32
    table = tables([1] * B, B, 1, g)
    q, k, v = torch.zeros(B, 2, d), torch.zeros(B, page, 2, d), torch.ones(B, page, 2, d)
    q[:, :, 0] = 1
    k[:, 1, :, 0] = -torch.linspace(85, 124.5, B)[:, None] * float(np.log(2))
    v[:, 1, :, ::2] = float("inf")
    lengths = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    out = dcn.paged_attention(*(a.bfloat16().cuda() for a in (q, k, v)), table, lengths, scale=1.0)
    assert torch.all(out[..., ::2] == float("inf")) and torch.all(out[..., 1::2] == 1)
