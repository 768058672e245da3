"""dcn_group_norm and its backward (through the binding) against the definition in 64 bits,
element by element, within the bounds that norm_oracle derives from the stated arithmetic."""

import zlib

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
import norm_oracle
from attention_oracle import check

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# name: shape (channels last), groups, weight and bias, mean of the values
CASES = {
    "c5": ((1, 25, 42, 256), 32, True, 0.0),
    "c4_batch2": ((2, 50, 84, 256), 32, True, 0.0),
    "one_position": ((3, 64), 4, True, 0.0),
    "two_positions": ((2, 2, 48), 3, True, 0.0),
    "one_value": ((2, 1, 16), 16, True, 0.0),                # a group of one value: its own mean, variance 0
    "one_group": ((2, 11, 13, 24), 1, True, 0.0),
    "a_channel_each": ((2, 9, 31, 40), 40, True, 0.0),       # instance normalisation
    "odd_channels": ((2, 17, 19, 81), 27, True, 0.0),        # rows start anywhere
    "one_channel": ((2, 37, 1), 1, True, 0.0),
    "no_parameters": ((2, 15, 14, 96), 8, False, 0.0),
    "long_rows": ((1, 7, 5, 4136), 8, True, 0.0),            # more vectors in a row than threads (fp32)
    "most_channels": ((1, 6, 8192), 512, True, 0.0),
    "odd_long_rows": ((1, 40, 1001), 7, True, 0.0),
    "groups_600": ((1, 33, 1200), 600, True, 0.0),           # more groups than threads
    "far_mean": ((2, 40, 31, 64), 8, True, 300.0),           # the variance is no difference of large sums
    "large": ((1, 100, 168, 64), 16, True, 1.0),
    "batch_9": ((9, 30, 41, 32), 4, True, 0.0),
}
ACTS = ["none", "relu", "silu", "gelu"]


def make(name, dtype, act):
    shape, G, params, mean = CASES[name]
    g = torch.Generator().manual_seed(zlib.crc32(f"{name} {act}".encode()))
    t = DT[dtype]
    C = shape[-1]
    x = torch.randn(shape, generator=g) * (0.5 + torch.rand(C, generator=g)) + torch.randn(C, generator=g) * 0.5 + mean
    w = (1 + 0.3 * torch.randn(C, generator=g)).to(t).cuda() if params else None
    b = (0.3 * torch.randn(C, generator=g)).to(t).cuda() if params else None
    go = torch.randn(shape, generator=g).to(t).cuda()
    return x.to(t).cuda(), G, w, b, go


def f64(t):
    return None if t is None else t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_norm_and_gradients(name, dtype):
    for act in ACTS if name in ("c5", "odd_channels") else [ACTS[zlib.crc32(name.encode()) % 4]]:
        print(f"[gpu-test] norm {name} {dtype} {act}", flush=True)
        x, G, w, b, go = make(name, dtype, act)
        out, mean, rstd = dcn.group_norm_act(x, G, w, b, eps=1e-5, activation=act, return_stats=True)
        torch.cuda.synchronize()
        ref = norm_oracle.forward(f64(x), G, f64(w), f64(b), float(np.float32(1e-5)), act, dtype)
        for n, t in (("mean", mean), ("rstd", rstd), ("out", out)):
            check(f64(t), ref[n], ref[n + "_tol"], f"{act} {n}")
        assert torch.equal(dcn.group_norm_act(x, G, w, b, eps=1e-5, activation=act), out)
        grads = dcn.group_norm_act_backward(go, x, mean, rstd, G, w, b, activation=act)
        torch.cuda.synchronize()
        ref = norm_oracle.backward(f64(go), f64(x), f64(mean), f64(rstd), G, f64(w), f64(b), act, dtype)
        for n, t in zip(("gx", "gw", "gb"), grads):
            if t is not None:
                check(f64(t), ref[n], ref[n + "_tol"], f"{act} {n}")
        assert (grads[1] is None) == (w is None)
        again = dcn.group_norm_act_backward(go, x, mean, rstd, G, w, b, activation=act)
        assert all(s is None or torch.equal(s, t) for s, t in zip(grads, again)), "the same call gave other bits"


@pytest.mark.parametrize("hw", [(25, 42), (70, 90)])   # in a workgroup's registers, and in two passes
@pytest.mark.parametrize("where", ["first", "last", "first channel"])
def test_a_position_far_out(hw, where):
    """One position 1e4 standard deviations out, wherever a sum about a sample could take it as its
    sample: squares are still summed about something near the mean, to ACC of the variance; the
    mean's error, ACC of the mean of |x|, is small against the standard deviation."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, *hw, 32)).astype(np.float32)
    if where == "first channel":
        x[:, 0, 0, ::8] = 1e4
    else:
        x[(slice(None), 0, 0) if where == "first" else (slice(None), -1, -1)] = 1e4
    out = dcn.group_norm_act(torch.from_numpy(x).cuda(), 4).double().cpu().numpy()
    g = x.astype(np.float64).reshape(2, -1, 4, 8)
    dev = g - g.mean((1, 3), keepdims=True)
    want = (dev / np.sqrt((dev ** 2).mean((1, 3), keepdims=True) + 1e-5)).reshape(x.shape)
    assert (np.abs(out - want) <= norm_oracle.ACC * (1 + np.abs(want))).all()


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gradients_against_differences(act):
    """<gradient, direction> against central differences of the definition in 64 bits."""
    x, G, w, b, go = make("no_parameters", "f32", act)
    w, b = (torch.linspace(0.5, 1.5, 96, device="cuda"), torch.linspace(-1, 1, 96, device="cuda"))
    _, mean, rstd = dcn.group_norm_act(x, G, w, b, activation=act, return_stats=True)
    grads = [f64(t) for t in dcn.group_norm_act_backward(go, x, mean, rstd, G, w, b, activation=act)]
    ref = norm_oracle.backward(f64(go), f64(x), f64(mean), f64(rstd), G, f64(w), f64(b), act, "f32")
    # the statistics that the call is given are rounded: their bound, carried into each gradient, is relative
    stats = norm_oracle.forward(f64(x), G, f64(w), f64(b), 1e-5, act, "f32")
    rel = float((stats["mean_tol"] * stats["rstd"] + stats["rstd_tol"] / stats["rstd"]).max())
    rng = np.random.default_rng(4)
    for i, name in enumerate(("gx", "gw", "gb")):
        base = [f64(x), f64(w), f64(b)]
        step, h, loss = rng.standard_normal(base[i].shape), 1e-5, []
        for sign in (1, -1):
            at = list(base)
            at[i] = base[i] + sign * h * step
            loss.append((norm_oracle.forward(at[0], G, at[1], at[2], 1e-5, act, "f32")["out"] * f64(go)).sum())
        diff = (loss[0] - loss[1]) / (2 * h)
        tol = (np.abs(step) * ref[name + "_tol"]).sum() + (10 * rel + 1e-6) * np.abs(step * ref[name]).sum()
        assert abs((grads[i] * step).sum() - diff) <= tol, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned_rows_and_in_place(dtype):
    """A map that starts 1 element into its buffer (no 16-byte rows), and out = input."""
    x, G, w, b, go = make("c5", dtype, "silu")
    out, mean, rstd = dcn.group_norm_act(x, G, w, b, activation="silu", return_stats=True)
    y = x.clone()
    assert dcn.group_norm_act(y, G, w, b, activation="silu", out=y) is y
    assert torch.equal(y, out)
    buf = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
    xu = buf[1:].view(x.shape)
    xu.copy_(x)
    ref = norm_oracle.forward(f64(x), G, f64(w), f64(b), float(np.float32(1e-5)), "silu", dtype)
    ou, mu, ru = dcn.group_norm_act(xu, G, w, b, activation="silu", return_stats=True)
    for n, t in (("mean", mu), ("rstd", ru), ("out", ou)):
        check(f64(t), ref[n], ref[n + "_tol"], n)
    ref = norm_oracle.backward(f64(go), f64(x), f64(mean), f64(rstd), G, f64(w), f64(b), "silu", dtype)
    for n, t in zip(("gx", "gw", "gb"), dcn.group_norm_act_backward(go, xu, mean, rstd, G, w, b, activation="silu")):
        check(f64(t), ref[n], ref[n + "_tol"], n)


def test_constant_input_and_not_finite():
    x = torch.full((2, 33, 8), 7.25, device="cuda")
    out, mean, rstd = dcn.group_norm_act(x, 2, return_stats=True)
    assert torch.all(out == 0) and torch.all(mean == 7.25)
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    x[1, 5, 3] = float("nan")
    out = dcn.group_norm_act(x, 2, activation="relu")
    assert torch.all(out[0] == 0) and torch.all(out[1, :, 4:] == 0) and torch.all(torch.isnan(out[1, :, :4]))


def test_empty_batch_and_only_the_gradients_asked_for():
    x = torch.empty((0, 4, 5, 16), device="cuda")
    w = torch.ones(16, device="cuda")
    out, mean, rstd = dcn.group_norm_act(x, 4, w, w, return_stats=True)
    assert out.shape == x.shape and mean.shape == (0, 4)
    gx, gw, gb = dcn.group_norm_act_backward(x, x, mean, rstd, 4, w, w)
    assert gx.shape == x.shape and torch.all(gw == 0) and torch.all(gb == 0)
    for name in ("c5", "large"):
        x, G, w, b, go = make(name, "bf16", "silu")
        _, mean, rstd = dcn.group_norm_act(x, G, w, b, return_stats=True)
        full = dcn.group_norm_act_backward(go, x, mean, rstd, G, w, b, activation="silu")
        desc = dcn.norm_desc(x, G, w, b, activation="silu")
        nb = dcn.dcn_group_norm_backward_workspace_bytes(desc)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        for wanted in ((0,), (1,), (2,), (0, 2)):
            got = [torch.empty_like(full[i]) if i in wanted else None for i in range(3)]
            dcn.dcn_group_norm_backward(desc, x, w, b, mean, rstd, go, *got, ws, nb)
            for i in wanted:
                assert torch.equal(got[i], full[i])


def test_addresses_beyond_32_bits():
    """A map of more than 2^31 elements: its last rows, against the same values alone."""
    C, P = 64, (1 << 25) + 1000
    x = torch.zeros((1, P, C), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    x[0, -500:] = torch.randn((500, C), generator=g).to(torch.bfloat16).cuda()
    out, mean, rstd = dcn.group_norm_act(x, 8, return_stats=True)
    tail = f64(x[0, -500:]).reshape(500, 8, 8)
    N = P * 8
    m = tail.sum((0, 2)) / N
    v = (tail ** 2).sum((0, 2)) / N - m * m
    want = ((tail - m[None, :, None]) / np.sqrt(v + 1e-5)[None, :, None]).reshape(500, C)
    # sums of 500 * 8 values among zeros, 8 sqrt(n) u; bf16 output
    tol = 2.0 ** -8 * np.abs(want) + 8 * np.sqrt(4096.0) * 2.0 ** -24 * (np.abs(want) + 1)
    check(f64(out[0, -500:]), want, tol, "out")


def test_on_a_side_stream_and_in_a_graph():
    for name in ("c5", "large"):
        x, G, w, b, go = make(name, "bf16", "silu")

        def both():
            out, mean, rstd = dcn.group_norm_act(x, G, w, b, activation="silu", return_stats=True)
            return (out, mean, rstd) + dcn.group_norm_act_backward(go, x, mean, rstd, G, w, b, activation="silu")

        want = both()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = both()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(s, t) for s, t in zip(want, got))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = both()
        torch.cuda.synchronize()
        x0 = x.clone()
        for f in (1.0, -0.5, 2.0):
            x.copy_((x0.float() * f + f).to(x0.dtype))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(s, t) for s, t in zip(both(), got)), name
        del graph


def test_refusals():
    x, G, w, b, go = make("c5", "f32", "silu")
    f = dcn.group_norm_act
    with pytest.raises(TypeError):
        f(x.double(), G)
    for bad in (dict(activation="tanh"), dict(weight=w[:5]), dict(weight=w.bfloat16()), dict(bias=b.cpu())):
        with pytest.raises(ValueError):
            f(x, G, **bad)
    for bad in (x[:, :, ::2], x.permute(0, 3, 1, 2), x[0, 0, 0], x.cpu()):
        with pytest.raises(ValueError):
            f(bad, G)
    for groups, eps in ((0, 1e-5), (3, 1e-5), (-4, 1e-5), (G, -1.0), (G, float("nan"))):
        with pytest.raises(dcn.DcnError) as e:
            f(x, groups, eps=eps)
        assert e.value.status == dcn.E_ARG
    with pytest.raises(dcn.DcnError) as e:
        f(torch.zeros((1, 2, 8200), device="cuda"), 4)
    assert e.value.status == dcn.E_UNSUPPORTED
    _, mean, rstd = f(x, G, return_stats=True)
    for bad in ((go[:, 1:], mean, rstd), (go.bfloat16(), mean, rstd), (go, mean[:, 1:], rstd), (go, mean, rstd.double())):
        with pytest.raises(ValueError):
            dcn.group_norm_act_backward(bad[0], x, bad[1], bad[2], G, w, b)
