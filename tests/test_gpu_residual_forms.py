"""The joins' forms that test_gpu_residual has at narrow rows only: no branch norm, gate or scale, no next norm, a
scale or a gate without a branch norm, at rows of several waves, whole and not, and beyond 4096 channels."""

import pytest
import torch

import deformable_convolution_vision_amd as dcn
import test_gpu_residual as base

pytestmark = pytest.mark.gpu

# name: shape, branch norm, next norm, gate, scale, weights and biases
CASES = {f"bare_{c}_{n}": ((2, 150, c), "none", n, None, False, True)
         for c in (5, 81, 513, 1030, 2040, 4096, 5001, 8192) for n in ("layer", "rms")}
CASES.update({f"no_next_{c}_{gate}": ((2, 150, c), n, "none", gate, gate is None, True)
              for c in (1030, 5001, 8192) for n, gate in (("layer", None), ("rms", "batch"), ("layer", "full"))})
CASES.update({f"no_branch_norm_{c}_{gate}": ((2, 150, c), "none", n, gate, gate is None, True)
              for c in (1030, 5001, 8192) for n, gate in (("layer", None), ("rms", "batch"), ("layer", "full"))})
CASES.update({f"sum_{c}": ((2, 40, c), "none", "none", None, False, False) for c in (81, 1030, 8192)})
CASES.update({f"scaled_sum_{c}": ((2, 40, c), "none", "none", "batch", True, False) for c in (81, 1030, 8191)})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_form_and_gradients(name, dtype, monkeypatch):
    print(f"[gpu-test] join form {name} {dtype}", flush=True)
    monkeypatch.setitem(base.CASES, name, CASES[name])
    x, y, go, gn, how = base.make(name, dtype)
    out, nxt, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    base.check_all((("out", out), ("next", nxt), ("stats", stats)), base.reference(x, y, how, dtype), name)
    grads = dcn.residual_norm_backward(go, gn, x, y, stats, **how)
    base.check_all(zip(base.NAMES, grads), base.gradient_reference(go, gn, x, y, stats, how, dtype), name)
    again = dcn.residual_norm_backward(go, gn, x, y, stats, **how)
    assert all(s is None or torch.equal(s, t) for s, t in zip(grads, again)), "the same call gave other bits"


@pytest.mark.parametrize("name", ["bare_8192_layer", "bare_1030_rms", "no_next_8192_None", "no_branch_norm_5001_full",
                                  "no_branch_norm_8192_batch"])
def test_only_the_gradients_asked_for(name, monkeypatch):
    monkeypatch.setitem(base.CASES, name, CASES[name])
    x, y, go, gn, how = base.make(name, "bf16")
    _, _, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    full = dcn.residual_norm_backward(go, gn, x, y, stats, **how)
    desc = dcn.residual_desc(x, y, **how)
    nb = dcn.dcn_residual_norm_backward_workspace_bytes(desc)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    ins = (x, y, how["gate"], how["scale"], how["branch_weight"], how["branch_bias"], how["next_weight"], stats)
    there = [i for i in range(8) if full[i] is not None]
    for wanted in [(i,) for i in there] + [tuple(there[1:])]:
        got = [torch.empty_like(full[i]) if i in wanted else None for i in range(8)]
        dcn.dcn_residual_norm_backward(desc, *ins, go, gn, *got, ws, nb)
        assert all(g is None or torch.equal(g, full[i]) for i, g in enumerate(got)), wanted
