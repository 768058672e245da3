"""The decoder example: its step's loss and gradients against autograd in 64 bits on the CPU (from
the layer's own output on, whose parity other tests hold), its single-token reader, and its training."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("deformable_decoder", os.path.join(ROOT, "examples", "deformable_decoder.py"))


@pytest.fixture(scope="module")
def example():
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def problem(example, dtype):
    cfg = example.Config(channels=64, heads=4, key_heads=2, head_dim=24, groups=8)
    p = example.init(cfg, dtype, "cuda", seed=3)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(2, 64, 18, 26, generator=gen).to(dtype).cuda()
    queries, target = (torch.randn(2, 11, 64, generator=gen).to(dtype).cuda() for _ in range(2))
    key_mask = torch.ones(2, 9, 13, dtype=torch.bool)
    key_mask[1, :, 8:] = False
    return cfg, p, x, queries, target, key_mask.view(2, -1).cuda()


def plain(cfg, p, z, queries, target, key_mask):
    """Loss and gradients from the layer's output z [B,Ho,Wo,C] on, by autograd in 64 bits."""
    names = ("norm_weight", "norm_bias", "q", "kv", "out")
    w = {n: p[n].double().cpu().requires_grad_() for n in names}
    z = z.double().cpu().requires_grad_()
    B, C, L = z.shape[0], cfg.channels, z.shape[1] * z.shape[2]
    t = z.reshape(B, L, cfg.groups, C // cfg.groups)
    n = (t - t.mean((1, 3), keepdim=True)) / (t.var((1, 3), unbiased=False, keepdim=True) + 1e-5).sqrt()
    tokens = torch.nn.functional.silu(n.reshape(B, L, C) * w["norm_weight"] + w["norm_bias"])
    kv = (tokens @ w["kv"]).view(B, L, 2, cfg.key_heads, 1, cfg.head_dim)
    key, value = (kv[:, :, i].expand(-1, -1, -1, cfg.heads // cfg.key_heads, -1).reshape(B, L, cfg.heads, -1)
                  for i in range(2))
    q = (queries.double().cpu() @ w["q"]).view(B, -1, cfg.heads, cfg.head_dim)
    s = torch.einsum("bqhd,bkhd->bhqk", q, key) * cfg.head_dim ** -0.5
    s = s.masked_fill(~key_mask.cpu()[:, None, None, :], -float("inf"))
    answer = torch.einsum("bhqk,bkhd->bqhd", s.softmax(-1), value).reshape(B, -1, cfg.width) @ w["out"]
    loss = 0.5 * (answer - target.double().cpu()).square().mean()
    loss.backward()
    return loss.item(), answer.detach(), z.grad, {n: w[n].grad for n in names}


# fp32: a chain of four stages, each with sums of at most 512 terms that are rounded by 2^-24 of the
# largest partial sum; later stages (weights of norm about 1) may raise what an earlier one left by
# 8 in all: 4 * 512 * 8 * 2^-24 = 1e-3 of the largest magnitude of a result.
TOL = 4 * 512 * 8 * 2.0 ** -24


def close(got, want):
    assert (got.double().cpu() - want).abs().max().item() <= TOL * want.abs().max().item()


def test_step_against_autograd(example):
    cfg, p, x, queries, target, key_mask = problem(example, torch.float32)
    loss, grads = example.step(cfg, p, x, queries, target, key_mask)
    y, offset, mask = example.dcn.deform_conv2d_layer(x, p["om_weight"], p["om_bias"], p["conv_weight"], p["conv_bias"],
                                                      stride=cfg.stride, padding=1)
    want, _, g_z, g_w = plain(cfg, p, y.permute(0, 2, 3, 1), queries, target, key_mask)
    assert abs(loss.item() - want) <= TOL * abs(want)
    for name, g in g_w.items():
        close(grads[name], g)
    # what the norm's backward hands on: the layer's bias gradient is its sum over positions
    close(grads["conv_bias"], g_z.sum((0, 1, 2)))


def test_reader_gives_the_decoders_rows(example):
    cfg, p, x, queries, target, key_mask = problem(example, torch.float32)
    y, _, _ = example.dcn.deform_conv2d_layer(x, p["om_weight"], p["om_bias"], p["conv_weight"], p["conv_bias"],
                                              stride=cfg.stride, padding=1)
    _, answer, _, _ = plain(cfg, p, y.permute(0, 2, 3, 1), queries, target, key_mask)
    reader = example.Reader(cfg, p, x, key_mask)
    for t in (0, 7):
        close(reader.token(queries[:, t]), answer[:, t])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_lower_the_loss(example, dtype):
    cfg, p, x, queries, target, key_mask = problem(example, dtype)
    losses = []
    for _ in range(8):
        loss, grads = example.step(cfg, p, x, queries, target, key_mask)
        losses.append(loss.item())
        for name in ("out", "q", "kv", "norm_weight", "norm_bias", "conv_weight", "conv_bias"):
            assert torch.isfinite(grads[name].float()).all(), name
            p[name] = (p[name].float() - 1.0 * grads[name].float()).to(dtype)
    assert losses[-1] < losses[0]
