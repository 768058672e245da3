"""dcn_rotary and its backward (through the binding) against the definition in 64 bits, element by
element, within the bounds that rotary_oracle derives from the stated arithmetic."""

import zlib

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
import rotary_oracle
from attention_oracle import check

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LAYOUTS = ["halves", "adjacent", "blocks"]

# name: B, L, H, D, sections, positions
CASES = {
    "one_token": (1, 1, 1, 64, (32,), "int"),
    "two_elements": (2, 3, 1, 2, (1,), "int"),
    "map": (2, 1050, 8, 32, (8, 8), "int"),
    "points": (2, 300, 8, 32, (8, 8), "float"),
    "clip_and_rest": (2, 77, 3, 64, (8, 8, 8), "int"),
    "four_axes": (1, 65, 5, 48, (5, 7, 3, 9), "float"),
    "uneven": (3, 33, 2, 40, (13, 7), "float"),
    "odd_head": (2, 29, 3, 37, (17,), "int"),
    "width_4": (2, 19, 4, 40, (12, 8), "float"),
    "width_2": (2, 19, 4, 20, (6, 4), "float"),
    "far": (1, 40, 2, 64, (32,), "far"),
    "many_heads": (1, 9, 37, 128, (64,), "int"),
    "one_row_of_many_heads": (1, 1, 300, 64, (16, 16), "float"),
    "widest_heads": (1, 3, 2, 512, (250,), "int"),
    "batch_33": (33, 7, 2, 32, (10,), "int"),
}


def make(name, dtype):
    B, L, H, D, sections, kind = CASES[name]
    g = torch.Generator().manual_seed(zlib.crc32(name.encode()))
    t = DT[dtype]
    x, go = (torch.randn((B, L, H, D), generator=g).to(t).cuda() for _ in range(2))
    axes = len(sections)
    if kind == "float":
        pos = (torch.rand((B, L, axes), generator=g) * 200 - 50).cuda()
    else:
        most = 1 << 30 if kind == "far" else 170
        pos = torch.randint(-5, most, (B, L, axes), generator=g, dtype=torch.int32).cuda()
    freq = torch.cat([100.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections]).float().cuda()
    return x, pos, freq, sections, go


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_rotation_and_gradients(name, dtype):
    for layout in LAYOUTS:
        print(f"[gpu-test] rotary {name} {dtype} {layout}", flush=True)
        x, pos, freq, sections, go = make(name, dtype)
        out = dcn.rotary_positions(x, pos, freq, sections, layout)
        torch.cuda.synchronize()
        how = (f64(pos), f64(freq), sections, layout)
        want, tol = rotary_oracle.rotate(f64(x), *how, dtype)
        check(f64(out), want, tol, f"{layout} out")
        gx, gp = dcn.rotary_positions_backward(go, pos, freq, sections, layout, input=x)
        torch.cuda.synchronize()
        want, tol = rotary_oracle.rotate(f64(go), *how, dtype, sign=-1)
        check(f64(gx), want, tol, f"{layout} grad_x")
        assert gp.dtype == torch.float32
        check(f64(gp), *rotary_oracle.position_gradients(f64(go), f64(x), *how), f"{layout} grad_positions")
        assert torch.equal(dcn.rotary_positions_backward(go, pos, freq, sections, layout), gx)
        again = dcn.rotary_positions_backward(go, pos, freq, sections, layout, input=x)
        assert torch.equal(again[0], gx) and torch.equal(again[1], gp), "the same call gave other bits"


def test_gradients_against_differences():
    """<gradient, direction> against central differences of the definition in 64 bits; angles up to
    170, so that a difference's h^2 term is below 1e-10 of the sum's terms."""
    for layout in LAYOUTS:
        x, pos, freq, sections, go = make("four_axes", "f32")
        gx, gp = (f64(t) for t in dcn.rotary_positions_backward(go, pos, freq, sections, layout, input=x))
        rng, h = np.random.default_rng(1), 1e-5
        base = [f64(x), f64(pos)]
        tols = [rotary_oracle.rotate(f64(go), f64(pos), f64(freq), sections, layout, "f32", sign=-1)[1],
                rotary_oracle.position_gradients(f64(go), f64(x), f64(pos), f64(freq), sections, layout)[1]]
        for i, grad in enumerate((gx, gp)):
            step, loss = rng.standard_normal(base[i].shape), []
            for sign in (1, -1):
                at = list(base)
                at[i] = base[i] + sign * h * step
                loss.append((rotary_oracle.rotate(at[0], at[1], f64(freq), sections, layout, "f32")[0] * f64(go)).sum())
            diff = (loss[0] - loss[1]) / (2 * h)
            size = np.abs(f64(go)).sum() * np.abs(f64(x)).max()
            assert abs((grad * step).sum() - diff) <= (np.abs(step) * tols[i]).sum() + 1e-8 * size, (layout, i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_alignment_and_in_place(dtype):
    x, pos, freq, sections, go = make("map", dtype)
    B, L, H, D = x.shape
    want = dcn.rotary_positions(x, pos, freq, sections)
    packed = torch.zeros((B, L, 3, H, D), dtype=x.dtype, device="cuda")
    packed[:, :, 1] = x
    assert torch.equal(dcn.rotary_positions(packed[:, :, 1], pos, freq, sections), want)     # a fused projection's slice
    first = x.transpose(1, 2).contiguous().transpose(1, 2)                                   # heads before positions
    assert torch.equal(dcn.rotary_positions(first, pos, freq, sections), want)
    assert torch.equal(dcn.rotary_positions(x[:1].expand(B, -1, -1, -1), pos, freq, sections),
                       dcn.rotary_positions(x[:1].repeat(B, 1, 1, 1), pos, freq, sections))  # a batch stride of 0
    shared = pos[:1].expand(B, -1, -1)
    assert torch.equal(dcn.rotary_positions(x, shared, freq, sections),
                       dcn.rotary_positions(x, shared.contiguous(), freq, sections))
    for shift in (1, 2, 4):                                                                  # rows that start off 16 bytes
        buf = torch.zeros(x.numel() + 8, dtype=x.dtype, device="cuda")
        xs = buf[shift:shift + x.numel()].view(x.shape)
        xs.copy_(x)
        assert torch.equal(dcn.rotary_positions(xs, pos, freq, sections), want)
        gx, gp = dcn.rotary_positions_backward(go, pos, freq, sections, input=xs)
        gx2, gp2 = dcn.rotary_positions_backward(go, pos, freq, sections, input=x)
        assert torch.equal(gx, gx2)
        tol = rotary_oracle.position_gradients(f64(go), f64(x), f64(pos), f64(freq), sections, "halves")[1]
        check(f64(gp), f64(gp2), 2 * tol, "grad_positions")
    y = x.clone()
    assert dcn.rotary_positions(y, pos, freq, sections, out=y) is y
    assert torch.equal(y, want)


def test_shared_positions_and_only_the_gradients_asked_for():
    x, pos, freq, sections, go = make("points", "bf16")
    shared = pos[:1].expand(x.shape[0], -1, -1)
    gx, gp = dcn.rotary_positions_backward(go, shared, freq, sections, input=x)
    gx2, gp2 = dcn.rotary_positions_backward(go, shared.contiguous(), freq, sections, input=x)
    assert torch.equal(gx, gx2) and torch.equal(gp, gp2)      # every repetition has its own
    desc = dcn.rotary_desc(x, pos, freq, sections)
    gx, gp = dcn.rotary_positions_backward(go, pos, freq, sections, input=x)
    only = torch.empty_like(gp)
    dcn.dcn_rotary_backward(desc, go, pos, freq, x, None, only)
    assert torch.equal(only, gp)
    only = torch.empty_like(gx)
    dcn.dcn_rotary_backward(desc, go, pos, freq, None, only, None)
    assert torch.equal(only, gx)
    g = go.clone()
    dcn.dcn_rotary_backward(desc, g, pos, freq, x, g, gp)     # grad_x in grad_out's place
    assert torch.equal(g, gx)


def test_nothing_to_do_and_not_finite():
    freq = torch.ones(4, device="cuda")
    for shape in ((0, 5, 2, 16), (2, 0, 2, 16)):
        x = torch.empty(shape, device="cuda")
        pos = torch.empty(shape[:2] + (1,), device="cuda")
        assert dcn.rotary_positions(x, pos, freq, (4,)).shape == shape
        gx, gp = dcn.rotary_positions_backward(x, pos, freq, (4,), input=x)
        assert gx.shape == shape and gp.shape == pos.shape
    x, pos = torch.randn((2, 3, 2, 16), device="cuda"), torch.ones((2, 3, 1), device="cuda")
    want = dcn.rotary_positions(x, pos, freq, (4,))
    bad, p2 = x.clone(), pos.clone()
    bad[0, 1, 1, 0] = float("nan")
    p2[1, 2] = float("inf")
    out = dcn.rotary_positions(bad, p2, freq, (4,))
    assert torch.isnan(out[0, 1, 1, [0, 4]]).all() and torch.isnan(out[1, 2, :, :8]).all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[0, 1, 1, [0, 4]] = False
    keep[1, 2, :, :8] = False
    assert torch.equal(out[keep], want[keep])


def test_addresses_beyond_32_bits():
    step = 1 << 26
    buf = torch.empty(40 * step, dtype=torch.bfloat16, device="cuda")
    x, pos, freq, sections, go = make("many_heads", "bf16")
    far = buf.as_strided((1, 9, 4, 128), (0, 4 * step, step, 1))
    far.copy_(x[:, :, :4])
    assert torch.equal(dcn.rotary_positions(far, pos, freq, sections),
                       dcn.rotary_positions(x[:, :, :4].contiguous(), pos, freq, sections))


def test_on_a_side_stream_and_in_a_graph():
    x, pos, freq, sections, go = make("points", "bf16")

    def both():
        return (dcn.rotary_positions(x, pos, freq, sections),) + dcn.rotary_positions_backward(go, pos, freq, sections,
                                                                                                input=x)
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
    for f in (1.0, -0.5, 2.0):
        x.copy_((x.float() * f).to(x.dtype))
        pos.add_(f)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(both(), got))
    del graph


def test_refusals():
    x, pos, freq, sections, go = make("points", "f32")
    f = dcn.rotary_positions
    for bad in ((x.double(), pos, freq), (x, pos.double(), freq), (x, pos.long(), freq)):
        with pytest.raises(TypeError):
            f(*bad, sections)
    wide = torch.zeros(40, device="cuda")
    for bad in ((x[0], pos, freq), (x, pos[:, 1:], freq), (x, pos[..., :1], freq), (x, pos, freq[1:]), (x.cpu(), pos, freq),
                (x, pos.cpu(), freq), (x, pos, freq.cpu()), (x, pos, freq.double()), (x, pos, wide[::2][:16]),
                (x.transpose(2, 3).contiguous().transpose(2, 3), pos, freq),
                (x, pos.transpose(1, 2).contiguous().transpose(1, 2), freq)):
        with pytest.raises(ValueError):
            f(*bad, sections)
    for sections2, layout in (((), "halves"), ((16, 0), "halves"), ((16, 1), "halves"), (sections, "thirds"),
                              ((4, 4, 4, 2, 2), "halves")):
        with pytest.raises(ValueError):
            f(x, pos, freq, sections2, layout)
    wide = torch.zeros((2, 3, 1, 513), device="cuda")
    with pytest.raises(dcn.DcnError) as e:
        f(wide, torch.zeros((2, 3, 1), device="cuda"), freq, (16,))
    assert e.value.status == dcn.E_UNSUPPORTED
    with pytest.raises(ValueError):
        f(x, torch.zeros(x.shape[:2] + (1,), device="cuda"), torch.zeros(17, device="cuda"), (17,))
    with pytest.raises(ValueError):
        f(x, pos, freq, sections, out=torch.empty_like(x)[:, ::2])
    with pytest.raises(ValueError):
        dcn.rotary_positions_backward(go[:, ::2], pos[:, ::2], freq, sections)
    with pytest.raises(ValueError):
        dcn.rotary_positions_backward(go, pos, freq, sections, input=x[:1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_heads_and_rows_far_apart(dtype):
    """Strides at and beyond 2^24 elements, at which addresses are formed in other products: the same bits as dense."""
    g = torch.Generator().manual_seed(3)
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x = torch.randn((2, 5, 3, 24), generator=g).to(t).cuda()
    freq = torch.rand(12, generator=g).cuda()
    at = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5, 1)
    want = dcn.rotary_positions(x, at, freq, (12,))
    for step in ((1 << 24) - 1, 1 << 24, (1 << 24) + 8):
        flat = torch.empty(3 * step + 2 * 5 * 24, dtype=t, device="cuda")
        far = flat.as_strided((2, 5, 3, 24), (5 * 24, 24, step, 1))
        far.copy_(x)
        assert torch.equal(dcn.rotary_positions(far, at, freq, (12,)), want), step
        flat = torch.empty(5 * step + 2 * 3 * 24, dtype=t, device="cuda")
        far = flat.as_strided((2, 5, 3, 24), (3 * 24, step, 24, 1))
        far.copy_(x)
        assert torch.equal(dcn.rotary_positions(far, at, freq, (12,)), want), step
