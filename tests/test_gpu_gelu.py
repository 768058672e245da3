"""The gelu of group norm and its slope alone, over the whole range of arguments: with weights of 0
the activation's argument is the bias, exactly.  Against 64 bits, within what the kernel's formula
can lose: Phi(-|z|) is a product of t = 1 / (1 + a |z|), a polynomial in a |z| t and exp(-z^2 / 2).
With u = 2^-24, t carries 3 u (a product, a sum, a reciprocal of 1 unit in the last place), the
polynomial's argument 5 u of which at most 1.5 times enters, its steps 4 u, the exponential
1.5 z^2 u from the three roundings of its argument and 2 u of its own, the products 2 u, the
polynomial itself 0.5 u; gelu's last product 1 u: (24 + 1.5 z^2) u of the value.  For bf16 the
polynomial is off by 4.6e-6 (77 u) and takes t itself, whose error enters 3 times: (100 + 1.5 z^2) u."""

import numpy as np
import pytest
import torch
from scipy.special import ndtr

import deformable_convolution_vision_amd as dcn
from attention_oracle import E, U, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("positions", [3, 5000])   # in a workgroup's registers, and in two passes
def test_gelu_and_its_slope(positions, dtype):
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    C, G = 2048, 32
    z = torch.from_numpy(np.concatenate([np.linspace(-12, 12, C - 256), np.geomspace(1e-30, 1, 128),
                                         -np.geomspace(1e-30, 1, 128)])).to(t)
    g = torch.Generator().manual_seed(7)
    x = torch.randn((1, positions, C), generator=g).to(t).cuda()
    w, b = torch.zeros(C, dtype=t, device="cuda"), z.cuda()
    out, mean, rstd = dcn.group_norm_act(x, G, w, b, activation="gelu", return_stats=True)
    zz = z.double().numpy()
    tol = ({"f32": 24, "bf16": 100}[dtype] + 1.5 * zz * zz) * U
    # 1e-37: results below fp32's smallest normal number may be flushed
    want = zz * ndtr(zz)
    check(out.double().cpu().numpy()[0], np.broadcast_to(want, (positions, C)),
          (tol + E[dtype]) * np.abs(want) + 1e-37, "gelu")
    go = torch.zeros_like(x)
    go[0, positions // 2] = 1                          # the bias' gradient is then one slope
    gb = dcn.group_norm_act_backward(go, x, mean, rstd, G, w, b, activation="gelu")[2]
    term = np.abs(zz) * np.exp(-zz * zz / 2) / np.sqrt(2 * np.pi)
    want = ndtr(zz) + np.sign(zz) * term
    check(gb.double().cpu().numpy(), want, tol * (ndtr(zz) + term) + (E[dtype] + U) * np.abs(want) + 1e-37, "slope")


def test_gelu_at_infinity_and_nan():
    z = torch.tensor([float("inf"), float("nan"), 1e30, 3e38, -1e10, -1e30], device="cuda")
    out = dcn.group_norm_act(torch.randn((1, 4, 6), device="cuda"), 1, torch.zeros_like(z), z, activation="gelu")[0, 0]
    assert out[0] == float("inf") and torch.isnan(out[1]) and torch.equal(out[2:4], z[2:4]) and torch.all(out[4:] == 0)
