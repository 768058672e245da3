"""Calls of rotary positions, joins and the paged cache that dcn.h allows and that the other tests do not make: outputs
in the inputs' places at rows and heads that are no whole vectors, more workgroups than one launch takes, the
largest page, the most batch elements with a gate of their own, pages that several entries name."""

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
import test_gpu_paged_weights
import test_gpu_residual as join
import test_gpu_rotary as rotary
from attention_oracle import check
from test_gpu_paged import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(rotary.CASES))
def test_rotation_in_place(name, dtype):
    for layout in rotary.LAYOUTS:
        x, pos, freq, sections, go = rotary.make(name, dtype)
        want = dcn.rotary_positions(x, pos, freq, sections, layout)
        gx, gp = dcn.rotary_positions_backward(go, pos, freq, sections, layout, input=x)
        desc, g, p = dcn.rotary_desc(x, pos, freq, sections, layout), go.clone(), torch.empty_like(gp)
        dcn.dcn_rotary_backward(desc, g, pos, freq, x, g, p)
        assert torch.equal(g, gx) and torch.equal(p, gp), layout
        g = go.clone()
        dcn.dcn_rotary_backward(desc, g, pos, freq, None, g, None)
        assert torch.equal(g, gx), layout
        dcn.rotary_positions(x, pos, freq, sections, layout, out=x)
        assert torch.equal(x, want), layout


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["odd_channels", "row_of_two_waves", "odd_wide", "odd_wider", "wide_runs", "wide_runs_gated",
                                  "wide_runs_shared", "plain_sum", "few_channels"])
def test_join_in_place(name, dtype):
    x, y, go, gn, how = join.make(name, dtype)
    out, nxt, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    full = dcn.residual_norm_backward(go, gn, x, y, stats, **how)
    desc = dcn.residual_desc(x, y, **how)
    params = [how[k] for k in ("gate", "scale", "branch_weight", "branch_bias", "next_weight", "next_bias")]
    for places in ("out in x, next in branch", "out in branch"):
        a, b = x.clone(), y.clone()
        n = None if nxt is None else b if places.endswith("next in branch") else torch.empty_like(nxt)
        o = a if places.startswith("out in x") else b
        dcn.dcn_residual_norm(desc, a, b, *params, o, n, None)
        assert torch.equal(o, out) and (nxt is None or torch.equal(n, nxt)), places
    nb = dcn.dcn_residual_norm_backward_workspace_bytes(desc)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    g, h = go.clone(), None if gn is None else gn.clone()
    grads = [g, torch.empty_like(y) if h is None else h] + [None if t is None else torch.empty_like(t) for t in params]
    dcn.dcn_residual_norm_backward(desc, x, y, *params[:4], params[4], stats, g, h, *grads, ws, nb)
    assert all(t is None or torch.equal(s, t) for s, t in zip(grads, full))


def test_a_gate_of_as_many_batch_elements_as_there_may_be():
    g = torch.Generator().manual_seed(2)
    x, y, gate, go, gn = (torch.randn(s, generator=g).cuda() for s in ((65530, 1, 24), (65530, 1, 24), (65530, 24),
                                                                        (65530, 1, 24), (65530, 1, 24)))
    how = {"gate": gate, "scale": torch.rand(24, generator=g).cuda(), "branch_norm": "rms", "branch_weight": None,
           "branch_bias": None, "next_norm": "layer", "next_weight": None, "next_bias": None}
    out, nxt, stats = dcn.residual_norm(x, y, return_stats=True, **how)
    join.check_all((("out", out), ("next", nxt), ("stats", stats)), join.reference(x, y, how, "f32"), "many")
    grads = dcn.residual_norm_backward(go, gn, x, y, stats, **how)
    join.check_all(zip(join.NAMES, grads), join.gradient_reference(go, gn, x, y, stats, how, "f32"), "many")


@pytest.mark.parametrize("width", [1, 200])
def test_more_sequences_than_a_launch_takes(width):
    """2.4 million pairs of a sequence and a key head, of one part each (a short table) or dealt out from lists."""
    g = torch.Generator().manual_seed(width)
    B, hkv, d, page, pages = 300000, 8, 8, 16, 512
    k, v = (torch.randn((pages, page, hkv, d), generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn((B, hkv, d), generator=g).bfloat16().cuda()
    table = torch.randint(0, pages, (1, width), generator=g, dtype=torch.int32).expand(B, -1).cuda()
    table = table[:1].expand(B, -1)                       # every sequence's is the same memory
    lengths = torch.randint(0, page + 1, (B,), generator=g, dtype=torch.int32)
    sample = torch.cat((torch.tensor([0, 1, B - 2, B - 1]), torch.randint(0, B, (300,), generator=g)))
    lengths[sample[::9]] = torch.randint(1, width * page + 1, (len(sample[::9]),), generator=g, dtype=torch.int32)
    lengths = lengths.cuda()
    out, lse = dcn.paged_attention(q, k, v, table, lengths, return_lse=True)
    at = sample.cuda()
    want, tol, wl, tl = test_gpu_paged_weights.reference(q[at], k, v, table[at], lengths[at], "bf16", d ** -0.5)
    check(f64(out[at]), want, tol, "out")
    check(f64(lse[at]), wl, tl, "lse")
    # and all of them against the same call in two halves, whose parts may differ: two roundings, and the bound's share
    half = torch.cat([dcn.paged_attention(q[i:i + B // 2], k, v, table[i:i + B // 2], lengths[i:i + B // 2])
                      for i in (0, B // 2)])
    off = (half.float() - out.float()).abs()
    assert (off <= 2.0 ** -7 * out.float().abs() * 1.01 + 2.0 ** -18 * v.float().abs().max()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_largest_page(dtype):
    """One page of 2^31 - 65537 positions, which are the same few in memory: lengths that end anywhere."""
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator().manual_seed(8)
    n = (1 << 31) - 65537
    q, k, v = (torch.randn(s, generator=g).to(t).cuda() for s in ((3, 4, 32), (1, 1, 2, 32), (1, 1, 2, 32)))
    table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    lengths = torch.tensor([0, 77, 5000], dtype=torch.int32, device="cuda")
    out = dcn.paged_attention(q, k.expand(1, n, 2, 32), v.expand(1, n, 2, 32), table, lengths)
    # every position is the same: its value
    value = v[0, 0].repeat_interleave(2, 0).float()
    assert torch.all(out[0] == 0)
    tol = 2 * torch.finfo(t).eps * value.abs() + 2.0 ** -16 * value.abs()
    assert all(((out[b].float() - value).abs() <= tol).all() for b in (1, 2))


def test_pages_named_twice():
    """Two sequences over the same pages, and a page twice in one: read as often as it is named; an append's rows that
    name one row of the cache leave one of theirs there."""
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(s, generator=g).cuda() for s in ((2, 4, 64), (5, 16, 2, 64), (5, 16, 2, 64)))
    table = torch.tensor([[3, 1, 3, 3], [3, 1, 4, 0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([64, 50], dtype=torch.int32, device="cuda")
    out, lse = dcn.paged_attention(q, k, v, table, lengths, return_lse=True)
    want, tol, wl, tl = test_gpu_paged_weights.reference(q, k, v, table, lengths, "f32", 0.125)
    check(f64(out), want, tol, "out")
    check(f64(lse), wl, tl, "lse")
    rows = torch.randn((2, 1, 2, 64), generator=g).cuda()
    starts = torch.tensor([17, 17], dtype=torch.int32, device="cuda")      # both page 1, place 1
    before = k.clone()
    dcn.paged_append(rows, rows, k, v, table, starts)
    assert ((k[1, 1] == rows[0, 0]) | (k[1, 1] == rows[1, 0])).all()
    keep = torch.ones(5, 16, dtype=torch.bool, device="cuda")
    keep[1, 1] = False
    assert torch.equal(k[keep], before[keep]) and np.isfinite(f64(k)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_gradient_of_values_that_are_not_finite(dtype):
    """What is not finite in an axis's pairs reaches that position's gradient, and no other axis's, row's or head's."""
    for name in ("map", "four_axes", "width_4"):
        for layout in rotary.LAYOUTS:
            x, pos, freq, sections, go = rotary.make(name, dtype)
            want = dcn.rotary_positions_backward(go, pos, freq, sections, layout, input=x)[1]
            # the second axis's first pair
            pairs = rotary.rotary_oracle.pairs_of(sections, layout)
            axis, first, second = pairs[sections[0]]
            assert axis == 1
            for tensor, bad in ((x, float("inf")), (go, float("nan")), (x, float("nan"))):
                was = tensor[1 if len(x) > 1 else 0, 3, -1, first].clone()
                tensor[1 if len(x) > 1 else 0, 3, -1, first] = bad
                gp = dcn.rotary_positions_backward(go, pos, freq, sections, layout, input=x)[1]
                tensor[1 if len(x) > 1 else 0, 3, -1, first] = was
                hit = torch.zeros_like(gp, dtype=torch.bool)
                hit[1 if len(x) > 1 else 0, 3, 1] = True
                assert torch.equal(gp[~hit], want[~hit]) and not torch.isfinite(gp[hit]).any(), (name, layout, bad)
