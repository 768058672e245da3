"""dcn_residual_norm and its backward (through the binding) against the definition in 64 bits,
element by element, within the bounds that residual_oracle derives from the stated arithmetic."""

import zlib

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
import residual_oracle
from attention_oracle import check

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = float(np.float32(1e-5))

# name: shape, branch norm, next norm, gate (None, "batch", "full"), scale, weights and biases
CASES = {
    "one_row": ((1, 1, 256), "none", "layer", None, False, True),
    "queries": ((2, 300, 256), "layer", "layer", None, True, True),
    "gated": ((3, 77, 256), "layer", "layer", "batch", True, True),
    "gated_full": ((2, 45, 192), "rms", "rms", "full", True, True),
    "rms_then_layer": ((2, 45, 96), "rms", "layer", "batch", False, True),
    "no_next": ((2, 33, 64), "layer", "none", "batch", True, True),
    "plain_sum": ((2, 33, 64), "none", "none", None, False, False),
    "no_parameters": ((2, 33, 128), "layer", "rms", None, False, False),
    "few_channels": ((2, 50, 16), "layer", "layer", "full", True, True),
    "odd_channels": ((2, 41, 81), "layer", "layer", "batch", True, True),
    "even_channels": ((2, 41, 150), "rms", "layer", "full", True, True),
    "one_channel": ((2, 5, 1), "rms", "layer", None, True, True),
    "row_of_a_wave": ((2, 70, 512), "layer", "rms", "full", False, True),
    "row_of_two_waves": ((2, 70, 520), "layer", "layer", "batch", True, True),
    "odd_wide": ((3, 31, 1030), "rms", "rms", "full", False, True),
    "odd_wider": ((2, 9, 2047), "layer", "layer", "batch", True, True),
    "wide_512_threads": ((1, 9, 4096), "layer", "layer", "full", True, True),
    "most_channels": ((2, 3, 8192), "layer", "layer", "batch", True, True),
    "wide_runs": ((2, 300, 4100), "layer", "rms", None, True, True),     # several rows of 1024 threads in turn
    "wide_runs_gated": ((1, 517, 5001), "rms", "layer", "full", True, True),
    "wide_runs_shared": ((2, 300, 8192), "layer", "layer", "batch", True, True),
    "most_odd_channels": ((1, 3, 8191), "layer", "rms", "full", True, True),
    "map": ((2, 50, 84, 256), "layer", "layer", "batch", True, True),
    "batch_600": ((600, 3, 32), "layer", "layer", "batch", True, True),
}
NAMES = ("gx", "gy", "ggate", "gscale", "gw1", "gb1", "gw2", "gb2")


def make(name, dtype):
    shape, n1, n2, gate, scale, params = CASES[name]
    g = torch.Generator().manual_seed(zlib.crc32(name.encode()))
    t, C = DT[dtype], shape[-1]

    def normal(*s, std=1.0, mean=0.0):
        return (torch.randn(s, generator=g) * std + mean).to(t).cuda()

    x, y, go, gn = normal(*shape, std=2, mean=0.3), normal(*shape), normal(*shape), normal(*shape)
    how = {"gate": None if gate is None else normal(*((shape[0], C) if gate == "batch" else shape), std=0.5, mean=0.7),
           "scale": normal(C, std=0.3, mean=0.5) if scale else None, "branch_norm": n1, "next_norm": n2}
    for side, kind in (("branch", n1), ("next", n2)):
        how[side + "_weight"] = normal(C, std=0.3, mean=1) if params and kind != "none" else None
        how[side + "_bias"] = normal(C, std=0.3) if params and kind != "none" else None
    return x, y, go, gn if n2 != "none" else None, how


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def rows(a):
    return None if a is None else a.reshape(a.shape[0], -1, a.shape[-1])


def reference(x, y, how, dtype):
    a = {k: f64(v) if isinstance(v, torch.Tensor) else v for k, v in how.items()}
    gate = a["gate"] if a["gate"] is None or a["gate"].shape != tuple(x.shape) or x.ndim == 2 else rows(a["gate"])
    return residual_oracle.forward(rows(f64(x)), rows(f64(y)), gate, a["scale"], a["branch_norm"], a["branch_weight"],
                                   a["branch_bias"], a["next_norm"], a["next_weight"], a["next_bias"], EPS, dtype)


def gradient_reference(go, gn, x, y, stats, how, dtype):
    a = {k: f64(v) if isinstance(v, torch.Tensor) else v for k, v in how.items()}
    gate = a["gate"] if a["gate"] is None or a["gate"].shape != tuple(x.shape) or x.ndim == 2 else rows(a["gate"])
    return residual_oracle.backward(rows(f64(go)), rows(f64(gn)), rows(f64(x)), rows(f64(y)), rows(f64(stats)), gate,
                                    a["scale"], a["branch_norm"], a["branch_weight"], a["branch_bias"], a["next_norm"],
                                    a["next_weight"], dtype)


def check_all(pairs, ref, what):
    for n, t in pairs:
        if t is not None:
            check(f64(t).reshape(ref[n].shape), ref[n], ref[n + "_tol"], f"{what} {n}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_join_and_gradients(name, dtype):
    print(f"[gpu-test] join {name} {dtype}", flush=True)
    x, y, go, gn, how = make(name, dtype)
    out, nxt, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    torch.cuda.synchronize()
    check_all((("out", out), ("next", nxt), ("stats", stats)), reference(x, y, how, dtype), name)
    again = dcn.residual_norm(x, y, **how)
    assert torch.equal(again[0], out) and (nxt is None or torch.equal(again[1], nxt))
    grads = dcn.residual_norm_backward(go, gn, x, y, stats, **how)
    torch.cuda.synchronize()
    check_all(zip(NAMES, grads), gradient_reference(go, gn, x, y, stats, how, dtype), name)
    for t, v in zip(grads[2:], (how["gate"], how["scale"], how["branch_weight"], how["branch_bias"], how["next_weight"],
                                how["next_bias"])):
        assert (t is None) == (v is None) and (t is None or t.shape == v.shape)
    again = dcn.residual_norm_backward(go, gn, x, y, stats, **how)
    assert all(s is None or torch.equal(s, t) for s, t in zip(grads, again)), "the same call gave other bits"


@pytest.mark.parametrize("name", ["gated", "gated_full", "odd_wide", "no_next"])
def test_gradients_against_differences(name):
    """<gradient, direction> against central differences of the definition in 64 bits."""
    x, y, go, gn, how = make(name, "f32")
    _, _, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    grads = [f64(t) for t in dcn.residual_norm_backward(go, gn, x, y, stats, **how)]
    ref = gradient_reference(go, gn, x, y, stats, how, "f32")
    fwd = reference(x, y, how, "f32")
    # the statistics that the call is given are rounded: their bound, relative to the deviation
    r, tol = fwd["stats"], fwd["stats_tol"]
    rel = float(max((tol[..., i] * r[..., i + 1] + tol[..., i + 1] / r[..., i + 1]).max() for i in (0, 2)))
    rng, h = np.random.default_rng(2), 1e-5
    held = {"gx": "x", "gy": "y", "ggate": "gate", "gscale": "scale", "gw1": "branch_weight", "gb1": "branch_bias",
            "gw2": "next_weight", "gb2": "next_bias"}
    base = {"x": f64(x), "y": f64(y), **{k: f64(v) if isinstance(v, torch.Tensor) else v for k, v in how.items()}}
    for i, n in enumerate(NAMES):
        if grads[i] is None:
            continue
        step, loss = rng.standard_normal(grads[i].shape), []
        for sign in (1, -1):
            a = dict(base)
            a[held[n]] = base[held[n]] + sign * h * step
            f = residual_oracle.forward(a["x"], a["y"], a["gate"], a["scale"], a["branch_norm"], a["branch_weight"],
                                        a["branch_bias"], a["next_norm"], a["next_weight"], a["next_bias"], EPS, "f32")
            loss.append((f["out"] * f64(go)).sum() + (0 if gn is None else (f["next"] * f64(gn)).sum()))
        diff = (loss[0] - loss[1]) / (2 * h)
        bound = (np.abs(step) * ref[n + "_tol"].reshape(step.shape)).sum() + (20 * rel + 1e-6) * np.abs(step * grads[i]).sum()
        assert abs((grads[i] * step).sum() - diff) <= bound + 1e-9 * np.abs(f64(go)).sum(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned_rows_and_in_place(dtype):
    """Inputs that start 1 or 2 elements into their buffers, and outputs in the inputs' places."""
    x, y, go, gn, how = make("gated", dtype)
    out, nxt, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    ref = reference(x, y, how, dtype)
    for shift in (1, 2):
        buf = torch.empty(x.numel() + 2, dtype=x.dtype, device="cuda")
        xu = buf[shift:shift + x.numel()].view(x.shape)
        xu.copy_(x)
        o, n, s = dcn.residual_norm(xu, y, return_stats=True, **how)
        check_all((("out", o), ("next", n), ("stats", s)), ref, "unaligned")
        grads = dcn.residual_norm_backward(go, gn, xu, y, stats, **how)
        check_all(zip(NAMES, grads), gradient_reference(go, gn, x, y, stats, how, dtype), "unaligned")
    desc = dcn.residual_desc(x, y, **how)
    a, b = x.clone(), y.clone()
    dcn.dcn_residual_norm(desc, a, b, how["gate"], how["scale"], how["branch_weight"], how["branch_bias"],
                          how["next_weight"], how["next_bias"], a, b, None)      # out in x's place, next in branch's
    assert torch.equal(a, out) and torch.equal(b, nxt)


def test_only_the_gradients_asked_for():
    for name in ("gated", "gated_full", "queries"):
        x, y, go, gn, how = make(name, "bf16")
        _, _, stats = dcn.residual_norm(x, y, return_stats=True, **how)
        full = dcn.residual_norm_backward(go, gn, x, y, stats, **how)
        desc = dcn.residual_desc(x, y, **how)
        nb = dcn.dcn_residual_norm_backward_workspace_bytes(desc)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        ins = (x, y, how["gate"], how["scale"], how["branch_weight"], how["branch_bias"], how["next_weight"], stats)
        for wanted in [(i,) for i in range(8)] + [(0, 1), (0, 4, 7)]:
            got = [torch.empty_like(full[i]) if i in wanted and full[i] is not None else None for i in range(8)]
            dcn.dcn_residual_norm_backward(desc, *ins, go, gn, *got, ws, nb)
            assert all(g is None or torch.equal(g, full[i]) for i, g in enumerate(got)), (name, wanted)
        # no workspace without parameters' gradients; grad_x in grad_out's place, grad_branch in grad_next's
        a, b = go.clone(), gn.clone()
        dcn.dcn_residual_norm_backward(desc, *ins, a, b, a, b, *[None] * 6, None, 0)
        assert torch.equal(a, full[0]) and torch.equal(b, full[1])


def test_no_upstream_gradient_on_one_side():
    x, y, go, gn, how = make("gated", "f32")
    _, _, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    zero = torch.zeros_like(go)
    for a, b in ((None, gn), (go, None), (None, None)):
        got = dcn.residual_norm_backward(a, b, x, y, stats, **how)
        want = dcn.residual_norm_backward(zero if a is None else a, zero if b is None else b, x, y, stats, **how)
        assert all(torch.equal(s, t) for s, t in zip(got, want))


def test_constant_rows_and_not_finite():
    x, y = torch.full((2, 9, 64), 3.0, device="cuda"), torch.full((2, 9, 64), 0.25, device="cuda")
    out, nxt = dcn.residual_norm(x, y, branch_norm="layer")
    assert torch.equal(out, x) and torch.all(nxt == 0)      # a variance of 0: the rows' deviations from the mean are 0
    y[1, 4, 7] = float("nan")
    out, nxt = dcn.residual_norm(x, y, branch_norm="layer")
    bad = torch.zeros((2, 9), dtype=torch.bool, device="cuda")
    bad[1, 4] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], x[~bad]) and torch.isnan(nxt[bad]).all()
    assert torch.all(nxt[~bad] == 0)
    y[1, 4, 7] = float("inf")
    out, nxt = dcn.residual_norm(x, y)
    assert out[1, 4, 7] == float("inf") and torch.isnan(nxt[bad]).all()


def test_no_rows():
    w = torch.ones(32, device="cuda")
    for shape in ((0, 4, 32), (3, 0, 32)):
        x = torch.empty(shape, device="cuda")
        gate = torch.ones((shape[0], 32), device="cuda")
        how = dict(gate=gate, scale=w, branch_norm="layer", branch_weight=w, branch_bias=w, next_weight=w, next_bias=w)
        out, nxt, stats = dcn.residual_norm(x, x, return_stats=True, **how)
        assert out.shape == shape and stats.shape == shape[:2] + (4,)
        grads = dcn.residual_norm_backward(x, x, x, x, stats, **how)
        torch.cuda.synchronize()
        assert all(torch.all(t == 0) for t in grads[2:]) and grads[0].shape == shape


def test_addresses_beyond_32_bits():
    """More than 2^31 elements: the last rows against the same rows alone."""
    C, P = 64, (1 << 25) + 1000
    x = torch.zeros((1, P, C), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    tail = torch.randn((2, 1, 500, C), generator=g).to(torch.bfloat16).cuda()
    x[0, -500:] = tail[0, 0]
    y = torch.zeros_like(x)
    y[0, -500:] = tail[1, 0]
    how = dict(branch_norm="layer", next_norm="rms")
    out, nxt, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    o, n, s = dcn.residual_norm(tail[0], tail[1], return_stats=True, **how)
    assert torch.equal(out[:, -500:], o) and torch.equal(nxt[:, -500:], n) and torch.equal(stats[:, -500:], s)
    assert torch.all(out[:, :5] == 0)
    del nxt
    gx, gy, *_ = dcn.residual_norm_backward(out, x, x, y, stats, **how)
    gx2, gy2, *_ = dcn.residual_norm_backward(o, tail[0], tail[0], tail[1], s, **how)
    assert torch.equal(gx[:, -500:], gx2) and torch.equal(gy[:, -500:], gy2)


def test_on_a_side_stream_and_in_a_graph():
    for name in ("gated", "odd_wide"):
        x, y, go, gn, how = make(name, "bf16")

        def both():
            out, nxt, stats = dcn.residual_norm(x, y, return_stats=True, **how)
            return [t for t in (out, nxt, stats) + dcn.residual_norm_backward(go, gn, x, y, stats, **how) if t is not None]

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
        y0 = y.clone()
        for f in (1.0, -0.5, 2.0):
            y.copy_((y0.float() * f + f).to(y0.dtype))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(s, t) for s, t in zip(both(), got)), name
        del graph


def test_refusals():
    x, y, go, gn, how = make("gated", "f32")
    f = dcn.residual_norm
    C = x.shape[-1]
    with pytest.raises(TypeError):
        f(x.double(), y.double())
    for bad in ((x[:, ::2], y[:, ::2]), (x, y[:1]), (x, y.bfloat16()), (x.cpu(), y.cpu()), (x[0, 0], y[0, 0]),
                (x, y.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            f(*bad)
    w = how["next_weight"]
    for bad in (dict(gate=how["gate"][:, :5]), dict(gate=how["gate"][0]), dict(scale=w[:5]), dict(scale=w.bfloat16()),
                dict(next_weight=w.cpu()), dict(next_norm="batch"), dict(branch_norm=None), dict(branch_weight=w),
                dict(branch_bias=w), dict(next_norm="none", next_weight=w), dict(gate=how["gate"].t().contiguous().t())):
        with pytest.raises(ValueError):
            f(x, y, **bad)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(dcn.DcnError) as e:
            f(x, y, eps=eps)
        assert e.value.status == dcn.E_ARG
    big = torch.zeros((1, 2, 8200), device="cuda")
    with pytest.raises(dcn.DcnError) as e:
        f(big, big)
    assert e.value.status == dcn.E_UNSUPPORTED
    _, _, stats = f(x, y, return_stats=True, **how)
    for bad in ((go[:, 1:], gn, stats), (go, gn.bfloat16(), stats), (go, gn, stats[..., :2]), (go, gn, stats.double())):
        with pytest.raises(ValueError):
            dcn.residual_norm_backward(bad[0], bad[1], x, y, bad[2], **how)
