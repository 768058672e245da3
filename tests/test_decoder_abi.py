"""Host side of the rotary, block join and paged cache entry points: descriptor, pointer and workspace
checks.  No GPU: every call here returns before its first HIP call."""

import ctypes
import os

import pytest
import torch

import deformable_convolution_vision_amd as dcn

FAKE, WS = 0x10000, 0x20000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dcn.LIB_PATH):
        from deformable_convolution_vision_amd import build
        build.build()
    return dcn.load_library()


def filled(d, over):
    for n, v in over.items():
        field = getattr(type(d), n)
        if isinstance(v, tuple):
            v = type(getattr(d, n))(*v)
        assert field is not None
        setattr(d, n, v)
    return d


def rotary(**over):
    return filled(dcn.RotaryDesc(2, 300, 8, 32, (300 * 256, 256, 32), (600, 2), 2, (8, 8, 0, 0), 2, 0, dcn.BF16), over)


def residual(**over):
    return filled(dcn.ResidualDesc(2, 300, 256, 1e-5, 2, 2, 1, dcn.BF16, 0), over)


def append(**over):
    return filled(dcn.AppendDesc(2, 5, 8, 2, 32, 9, 16, 4, (1280, 256, 32), (320, 64, 32), (320, 64, 32),
                                 (1024, 64, 32), (1024, 64, 32), 4, (10, 2), 2, (8, 8, 0, 0), 0, 1, dcn.F32), over)


def paged(**over):
    return filled(dcn.PagedDesc(2, 8, 2, 32, 600, 16, 300, (256, 32), (1024, 64, 32), (1024, 64, 32), 300, 0.2, dcn.F32), over)


def run_rotary(lib, d, backward, x=FAKE, pos=FAKE, freq=FAKE, out=FAKE, x0=FAKE, gp=FAKE):
    r = ctypes.byref(d) if d is not None else None
    return lib.dcn_rotary_backward(r, x, pos, freq, x0, out, gp, None) if backward else \
        lib.dcn_rotary(r, x, pos, freq, out, None)


def run_join(lib, d, backward, x=FAKE, y=FAKE, gate=FAKE, out=FAKE, nxt=0x30000, stats=FAKE, ws=WS, nb=1 << 40, grads=None):
    r = ctypes.byref(d) if d is not None else None
    if backward:
        g = dict(gx=FAKE, gy=FAKE, ggate=FAKE, gscale=FAKE, gw1=FAKE, gb1=FAKE, gw2=FAKE, gb2=FAKE) if grads is None else grads
        g = [g.get(n) for n in ("gx", "gy", "ggate", "gscale", "gw1", "gb1", "gw2", "gb2")]
        return lib.dcn_residual_norm_backward(r, x, y, gate, FAKE, FAKE, FAKE, FAKE, stats, FAKE, FAKE, *g, ws, nb, None)
    return lib.dcn_residual_norm(r, x, y, gate, FAKE, FAKE, FAKE, FAKE, FAKE, out, nxt, stats, None)


def run_append(lib, d, **over):
    p = dict(q=FAKE, k=FAKE, v=FAKE, pos=FAKE, freq=FAKE, table=FAKE, starts=FAKE, counts=0x40000, qo=FAKE, kp=FAKE, vp=FAKE,
             lengths=0x50000)
    p.update(over)
    return lib.dcn_paged_append(ctypes.byref(d) if d is not None else None, *p.values(), None)


def run_paged(lib, d, **over):
    p = dict(q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lengths=FAKE, out=FAKE, lse=FAKE, ws=WS, nb=1 << 40)
    p.update(over)
    return lib.dcn_paged_attention(ctypes.byref(d) if d is not None else None, *p.values(), None)


def size(f, d):
    n = ctypes.c_size_t(12345)
    return f(ctypes.byref(d), ctypes.byref(n)), n.value


BAD_TURNS = [dict(sections=(8, 0, 0, 0)), dict(sections=(8, -1, 0, 0)), dict(sections=(9, 8, 0, 0)), dict(axes=5), dict(axes=-1),
             dict(layout=3), dict(layout=-1), dict(position_type=2), dict(position_stride=(-1, 2)), dict(position_stride=(0, -2))]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad", BAD_TURNS + [
    dict(batch=-1), dict(length=-1), dict(heads=0), dict(head_dim=0), dict(axes=0), dict(x_stride=(-1, 256, 32)),
    dict(x_stride=(0, 256, -1))], ids=str)
def test_rotary_descriptors(lib, bad, backward):
    assert run_rotary(lib, rotary(**bad), backward) == dcn.E_ARG


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad", [dict(dtype=7), dict(head_dim=65537), dict(batch=1 << 20, length=1 << 10),
                                 dict(length=1 << 31), dict(heads=1 << 31, length=1)], ids=str)
def test_rotary_unsupported(lib, bad, backward):
    assert run_rotary(lib, rotary(**bad), backward) == dcn.E_UNSUPPORTED


def test_rotary_pointers(lib):
    for n in ("x", "pos", "freq", "out"):
        assert run_rotary(lib, rotary(), False, **{n: None}) == dcn.E_ARG, n
    for n in ("x", "pos", "freq", "x0"):
        assert run_rotary(lib, rotary(), True, **{n: None}) == dcn.E_ARG, n
    assert run_rotary(lib, rotary(), True, out=None, gp=None) == dcn.OK        # no gradient asked for
    assert run_rotary(lib, None, False) == dcn.E_ARG and run_rotary(lib, None, True) == dcn.E_ARG
    for d in (rotary(batch=0), rotary(length=0)):
        for backward in (False, True):
            assert run_rotary(lib, d, backward, None, None, None, None, None, None) == dcn.OK


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(positions=-1), dict(channels=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(branch_norm=3), dict(branch_norm=-1), dict(next_norm=3), dict(next_norm=-1), dict(gate=3), dict(gate=-1)], ids=str)
def test_join_descriptors(lib, bad, backward):
    d = residual(**bad)
    assert run_join(lib, d, backward) == dcn.E_ARG
    assert size(lib.dcn_residual_norm_backward_workspace_bytes, d) == (dcn.E_ARG, 12345)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad", [dict(dtype=2), dict(channels=8193), dict(batch=1 << 16, positions=1 << 15, gate=0),
                                 dict(positions=1 << 31), dict(batch=1 << 16, positions=1)], ids=str)
def test_join_unsupported(lib, bad, backward):
    d = residual(**bad)
    assert run_join(lib, d, backward) == dcn.E_UNSUPPORTED
    assert size(lib.dcn_residual_norm_backward_workspace_bytes, d) == (dcn.E_UNSUPPORTED, 12345)


def test_join_pointers_and_workspace(lib):
    for n in ("x", "y", "gate", "out", "nxt"):
        assert run_join(lib, residual(), False, **{n: None}) == dcn.E_ARG, n
    assert run_join(lib, residual(), False, nxt=FAKE, out=FAKE) == dcn.E_ARG
    assert run_join(lib, residual(), False, stats=FAKE + 4) == dcn.E_ARG
    for n in ("x", "y", "gate", "stats"):
        assert run_join(lib, residual(), True, **{n: None}) == dcn.E_ARG, n
    assert run_join(lib, residual(), True, stats=FAKE + 8) == dcn.E_ARG
    # gradients of what is not there
    assert run_join(lib, residual(gate=0), True) == dcn.E_ARG
    for d, n in ((residual(branch_norm=0), "gw1"), (residual(branch_norm=0), "gb1"), (residual(next_norm=0), "gw2"),
                 (residual(next_norm=0), "gb2")):
        assert run_join(lib, d, True, grads={"gx": FAKE, n: FAKE}) == dcn.E_ARG, n
    assert run_join(lib, None, False) == dcn.E_ARG and run_join(lib, None, True) == dcn.E_ARG
    f = lib.dcn_residual_norm_backward_workspace_bytes
    assert f(ctypes.byref(residual()), None) == dcn.E_ARG and f(None, ctypes.byref(ctypes.c_size_t())) == dcn.E_ARG
    for gate in (0, 1, 2):
        rc, nb = size(f, residual(gate=gate))
        assert rc == dcn.OK and nb >= 5 * 256 * 4
        g = {"gscale": FAKE}
        assert run_join(lib, residual(gate=gate), True, ws=None, grads=g) == dcn.E_WORKSPACE
        assert run_join(lib, residual(gate=gate), True, nb=nb - 1, grads=g) == dcn.E_WORKSPACE
        assert run_join(lib, residual(gate=gate), True, ws=WS + 64, grads=g) == dcn.E_WORKSPACE
    for d in (residual(batch=0), residual(positions=0)):
        assert size(f, d) == (dcn.OK, 0)
        assert lib.dcn_residual_norm(ctypes.byref(d), *[None] * 12) == dcn.OK
        assert lib.dcn_residual_norm_backward(ctypes.byref(d), *[None] * 19, 0, None) == dcn.OK


@pytest.mark.parametrize("bad", BAD_TURNS + [
    dict(batch=-1), dict(length=-1), dict(query_heads=-1), dict(key_heads=0), dict(head_dim=0), dict(num_pages=-1),
    dict(page_size=0), dict(max_pages=-1), dict(table_stride=-1), dict(q_stride=(0, 0, -1)), dict(k_stride=(-1, 0, 0)),
    dict(v_stride=(0, -1, 0)), dict(key_page_stride=(-1, 0, 0)), dict(value_page_stride=(0, 0, -1))], ids=str)
def test_append_descriptors(lib, bad):
    assert run_append(lib, append(**bad)) == dcn.E_ARG


@pytest.mark.parametrize("bad", [dict(dtype=5), dict(head_dim=65537), dict(batch=1 << 20, length=1 << 10),
                                 dict(page_size=1 << 20, max_pages=1 << 11), dict(num_pages=1 << 31),
                                 dict(query_heads=1 << 31)], ids=str)
def test_append_unsupported(lib, bad):
    assert run_append(lib, append(**bad)) == dcn.E_UNSUPPORTED


def test_append_pointers(lib):
    for n in ("q", "k", "v", "freq", "table", "starts", "qo", "kp", "vp"):
        assert run_append(lib, append(), **{n: None}) == dcn.E_ARG, n
    for n in ("starts", "counts"):
        assert run_append(lib, append(), lengths={"starts": FAKE, "counts": 0x40000}[n]) == dcn.E_ARG, n
    assert run_append(lib, None) == dcn.E_ARG
    every = ("q", "k", "v", "pos", "freq", "table", "starts", "counts", "qo", "kp", "vp", "lengths")
    assert run_append(lib, append(batch=0), **dict.fromkeys(every)) == dcn.OK
    assert run_append(lib, append(length=0), lengths=None, q=None, k=None, v=None) == dcn.OK


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(query_heads=0), dict(key_heads=0), dict(key_heads=3), dict(head_dim=0), dict(num_pages=-1),
    dict(page_size=0), dict(max_pages=-1), dict(table_stride=-1), dict(q_stride=(-1, 0)), dict(q_stride=(0, -1)),
    dict(key_page_stride=(0, -1, 0)), dict(value_page_stride=(-1, 0, 0)), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf"))], ids=str)
def test_paged_descriptors(lib, bad):
    d = paged(**bad)
    assert run_paged(lib, d) == dcn.E_ARG
    assert size(lib.dcn_paged_attention_workspace_bytes, d) == (dcn.E_ARG, 12345)


@pytest.mark.parametrize("bad", [dict(dtype=5), dict(head_dim=129), dict(batch=1 << 30), dict(num_pages=1 << 31),
                                 dict(page_size=1 << 20, max_pages=1 << 11)], ids=str)
def test_paged_unsupported(lib, bad):
    d = paged(**bad)
    assert run_paged(lib, d) == dcn.E_UNSUPPORTED
    assert size(lib.dcn_paged_attention_workspace_bytes, d) == (dcn.E_UNSUPPORTED, 12345)


def test_paged_pointers_and_workspace(lib):
    for n in ("q", "kp", "vp", "table", "lengths", "out"):
        assert run_paged(lib, paged(), **{n: None}) == dcn.E_ARG, n
    assert run_paged(lib, None) == dcn.E_ARG
    f = lib.dcn_paged_attention_workspace_bytes
    assert f(ctypes.byref(paged()), None) == dcn.E_ARG and f(None, ctypes.byref(ctypes.c_size_t())) == dcn.E_ARG
    rc, nb = size(f, paged())
    assert rc == dcn.OK and nb > 0 and size(f, paged()) == (rc, nb)            # 4800 positions are split
    assert run_paged(lib, paged(), ws=None) == dcn.E_WORKSPACE
    assert run_paged(lib, paged(), nb=nb - 1) == dcn.E_WORKSPACE
    assert run_paged(lib, paged(), ws=WS + 128) == dcn.E_WORKSPACE
    assert size(f, paged(batch=0)) == (dcn.OK, 0)
    assert lib.dcn_paged_attention(ctypes.byref(paged(batch=0)), *[None] * 8, 0, None) == dcn.OK


def test_binding_refuses_what_is_not_on_a_gpu(lib):
    x, f = torch.zeros(1, 3, 2, 8), torch.zeros(4)
    with pytest.raises(ValueError):
        dcn.rotary_positions(x, torch.zeros(1, 3, 1), f, (4,))
    with pytest.raises(ValueError):
        dcn.residual_norm(x, x)
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        dcn.paged_append(x, x, x, x, ints[:, None], ints)
    with pytest.raises(ValueError):
        dcn.paged_attention(x[0, :1], x, x, ints[:, None], ints)
    for call in (lambda: dcn.rotary_positions(x.half(), torch.zeros(1, 3, 1), f, (4,)), lambda: dcn.residual_norm(x.half(), x.half()),
                 lambda: dcn.paged_attention(x[0, :1].half(), x, x, ints[:, None], ints)):
        with pytest.raises(TypeError):
            call()
