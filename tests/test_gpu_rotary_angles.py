"""The cosines and sines of rotary positions: pairs of (1, 0) turn into them as they are (1 c - 0 s and 0 c + 1 s),
so fp32 outputs are what the kernels multiply with.

They are rounded to fp32 once (half its spacing at the value, which numpy gives) and off by 2^-30 besides,
and by the angle's own error, 2^-51 of it."""

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn

pytestmark = pytest.mark.gpu


def angles(kind):
    g = np.random.default_rng(len(kind))
    pairs = 64
    if kind == "tokens":
        pos, freq = np.arange(-3000, 3000), 10000.0 ** (-np.arange(pairs) / pairs)
    elif kind == "points":
        pos, freq = g.uniform(-50, 200, 6000), 100.0 ** (-np.arange(pairs) / pairs)
    elif kind == "quarter turns":      # next to where the nearest quarter changes
        pos, freq = np.arange(-3000, 3000), np.full(pairs, np.pi / 4) * (1 + np.arange(-32, 32) * 2.0 ** -23)
    elif kind == "far":
        pos, freq = g.integers(-2 ** 31, 2 ** 31, 6000), 10000.0 ** (-np.arange(pairs) / pairs)
    else:                              # small
        pos, freq = g.uniform(-1, 1, 6000), 2.0 ** (-np.arange(pairs) / 2.0)
    whole = kind in ("tokens", "quarter turns", "far")
    return torch.tensor(pos, dtype=torch.int32 if whole else torch.float32), torch.tensor(freq).float()


@pytest.mark.parametrize("kind", ["tokens", "points", "quarter turns", "far", "small"])
def test_cosines_and_sines(kind):
    print(f"[gpu-test] angles {kind}", flush=True)
    pos, freq = angles(kind)
    n = len(freq)
    x = torch.cat((torch.ones(n), torch.zeros(n))).expand(1, len(pos), 1, 2 * n).contiguous().cuda()
    at = pos.view(1, -1, 1).cuda()
    out = dcn.rotary_positions(x, at, freq.cuda(), (n,))[0, :, 0].double().cpu().numpy()
    back = dcn.rotary_positions_backward(x, at, freq.cuda(), (n,))[0, :, 0].double().cpu().numpy()
    t = pos.double().numpy()[:, None].astype(np.longdouble) * freq.double().numpy()
    for got, want in ((out[:, :n], np.cos(t)), (out[:, n:], np.sin(t)), (back[:, :n], np.cos(t)), (back[:, n:], -np.sin(t))):
        half = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64) / 2
        off = np.abs(got - want.astype(np.float64))
        # (half of the spacing of the next binade where the value is just below it)
        half = np.maximum(half, np.spacing(np.abs(got).astype(np.float32)).astype(np.float64) / 2)
        assert np.all(off <= half + 2.0 ** -30 + 2.0 ** -51 * np.abs(t).astype(np.float64)), (kind, (off - half).max() * 2 ** 30)
    # appended keys are turned by the same
    if kind != "tokens":
        return
    keys = x[:, :2000].reshape(2, 1000, 1, 2 * n)
    kp, vp = (torch.zeros((20, 200, 1, 2 * n), device="cuda") for _ in range(2))
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    starts = torch.tensor([0, 7], dtype=torch.int32, device="cuda")
    dcn.paged_append(keys, keys, kp, vp, table, starts, frequencies=freq.cuda(), sections=(n,))
    rows = kp.view(2, 2000, 2 * n).double().cpu().numpy()
    for b, s in enumerate((0, 7)):
        assert np.array_equal(rows[b, s:s + 1000], out[3000 + s:4000 + s])
