"""More small problems than one dispatch counts threads for (2^32): group norm of many small maps,
against the definition in 64 bits."""

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
import norm_oracle
from attention_oracle import check

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
