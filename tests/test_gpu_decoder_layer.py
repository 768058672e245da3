"""The decoder layer example: its step's loss and every gradient against autograd in 64 bits on the CPU, and
its tokens against attention over all earlier ones, kept whole."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))


@pytest.fixture(scope="module")
def example():
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def problem(example, dtype):
    cfg = example.Config(channels=72, heads=4, key_heads=2, head_dim=24, hidden=96, page=8)
    p = example.init(cfg, dtype, "cuda", seed=5)
    gen = torch.Generator().manual_seed(6)
    size = (7, 9)

    def normal(*shape):
        return torch.randn(shape, generator=gen).to(dtype).cuda()

    content, embed, states, target = (normal(2, n, 72) for n in (13, 13, 63, 13))
    gate = (0.5 + 0.2 * normal(2, 72).float()).to(dtype)
    points = (torch.rand((2, 13, 2), generator=gen) * 7).cuda()
    return cfg, p, content, embed, points, gate, states, size, target


def turned(x, at, freq):
    """Rotation by rows and columns, each axis's block by halves, in 64 bits."""
    n, parts = freq.shape[0] // 2, []
    for axis in range(2):
        t = at[:, :, axis, None, None] * freq[axis * n:(axis + 1) * n]
        a, b = x[..., 2 * n * axis:2 * n * axis + n], x[..., 2 * n * axis + n:2 * n * (axis + 1)]
        parts += [a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()]
    return torch.cat(parts, -1)


def rms(x):
    return x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt()


def plain(example, cfg, p, content, embed, points, gate, states, size, target):
    held = {"content": content, "embed": embed, "points": points, "gate": gate, "states": states, **p}
    w = {n: t.double().cpu().requires_grad_() for n, t in held.items()}
    freq, at = example.frequencies(cfg, "cpu").double(), example.grid(*size, "cpu").double().expand(2, -1, -1)
    h0 = w["content"] + w["embed"]
    B, Lq, C = h0.shape
    q = (rms(h0) * w["embed_norm"] @ w["q"]).view(B, Lq, cfg.heads, -1)
    kv = (w["states"] @ w["kv"]).view(B, -1, 2, cfg.key_heads, cfg.head_dim)
    q, k = turned(q, w["points"], freq), turned(kv[:, :, 0], at, freq)
    share = cfg.heads // cfg.key_heads
    k, v = (t.repeat_interleave(share, 2) for t in (k, kv[:, :, 1]))
    s = torch.einsum("bqhd,bkhd->bhqk", q, k) * cfg.head_dim ** -0.5
    read = torch.einsum("bhqk,bkhd->bqhd", s.softmax(-1), v).reshape(B, Lq, -1)
    h1 = h0 + w["gate"][:, None] * w["read_scale"] * rms(read @ w["out"]) * w["read_norm"]
    d = h1 - h1.mean(-1, keepdim=True)
    n1 = d / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w["mid_norm"] + w["mid_bias"]
    h2 = h1 + w["ff_scale"] * (torch.relu(n1 @ w["up"]) @ w["down"])
    loss = 0.5 * (h2 - target.double().cpu()).square().mean()
    loss.backward()
    return loss.item(), {n: t.grad for n, t in w.items() if t.grad is not None}


# fp32: a chain of about ten stages, sums of at most 128 terms that are rounded by 2^-24 of the largest partial
# sum; the stages' Jacobians (weights of norm about 1, three norms of rows) may raise what an earlier one left by
# 16 in all: 10 * 128 * 16 * 2^-24 = 1.2e-3 of the largest magnitude of a result.
TOL = 10 * 128 * 16 * 2.0 ** -24


def test_loss_and_gradients(example):
    args = problem(example, torch.float32)
    loss, grads = example.step(*args)
    want_loss, want = plain(example, *args)
    assert abs(loss.item() - want_loss) <= TOL * want_loss
    assert set(grads) == set(want) and {"points", "gate", "states", "kv", "embed_norm"} <= set(want)
    for n, g in grads.items():
        off = (g.double().cpu() - want[n]).abs().max().item()
        assert off <= TOL * want[n].abs().max().item(), (n, off)


def test_runs_in_bf16(example):
    loss, grads = example.step(*problem(example, torch.bfloat16))
    assert torch.isfinite(loss) and all(torch.isfinite(g).all() for g in grads.values())
    assert all(g.dtype == (torch.float32 if n == "points" else torch.bfloat16) for n, g in grads.items())


def test_tokens_against_attention_over_all_of_them(example):
    """fp32, four stages: TOL's rule with 4 in place of 10 stages is within it."""
    cfg, p, content = problem(example, torch.float32)[:3]
    writer = example.Writer(cfg, p, 2, 24)
    counts = torch.tensor([9, 4], dtype=torch.int32, device="cuda")
    writer.append(content[:, :9], counts=counts)
    w = {n: t.double().cpu() for n, t in p.items()}
    past = [content[b, :int(counts[b])].double().cpu() for b in range(2)]
    freq = writer.freq.double().cpu()
    hidden = content[:, 9].contiguous()
    for _ in range(5):
        out = writer.token(hidden)
        for b in range(2):
            past[b] = torch.cat((past[b], hidden[b:b + 1].double().cpu()))
            n = past[b].shape[0]
            qkv = (past[b] @ w["self_qkv"]).view(n, cfg.heads + 2 * cfg.key_heads, cfg.head_dim)
            t = torch.arange(n, dtype=torch.float64)[:, None, None] * freq
            half = cfg.head_dim // 2
            turn = qkv[:, :cfg.heads + cfg.key_heads]
            x, y = turn[..., :half], turn[..., half:]
            turn = torch.cat((x * t.cos() - y * t.sin(), y * t.cos() + x * t.sin()), -1)
            q, k, v = turn[-1, :cfg.heads], turn[:, cfg.heads:], qkv[:, cfg.heads + cfg.key_heads:]
            share = cfg.heads // cfg.key_heads
            k, v = k.repeat_interleave(share, 1), v.repeat_interleave(share, 1)
            a = (torch.einsum("hd,khd->hk", q, k) * cfg.head_dim ** -0.5).softmax(-1)
            branch = torch.einsum("hk,khd->hd", a, v).reshape(-1) @ w["self_out"]
            want = past[b][-1] + rms(branch)
            assert (out[b].double().cpu() - want).abs().max() <= TOL * want.abs().max()
        hidden = out
    assert writer.lengths.tolist() == [14, 9]
    assert torch.equal(writer.lengths, counts + 5)


def test_main(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["decoder_layer.py", "--steps", "2"])
    example.main()
    assert "eight tokens after [48, 31]" in capsys.readouterr().out
