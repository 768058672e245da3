"""Host side of the cross attention entry points: descriptor, pointer and workspace checks.
No GPU: every call here returns before its first HIP call."""

import ctypes
import os

import pytest

import deformable_convolution_vision_amd as dcn


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dcn.LIB_PATH):
        from deformable_convolution_vision_amd import build
        build.build()
    return dcn.load_library()


def desc(**over):
    d = dcn.AttnDesc(2, 300, 4200, 8, 4, 32, (300 * 256, 256, 32), (4200 * 128, 128, 32), (4200 * 128, 128, 32), 4200,
                     0.2, dcn.BF16)
    for n, v in over.items():
        if n.endswith("_stride") and n != "mask_stride":
            v = (ctypes.c_int64 * 3)(*v)
        setattr(d, n, v)
    return d


FAKE, WS = 0x10000, 0x20000


def status(lib, d, backward, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, go=FAKE, ws=WS, nb=1 << 40):
    r = ctypes.byref(d) if d is not None else None
    if backward:
        return lib.dcn_cross_attention_backward(r, q, k, v, None, out, lse, go, FAKE, FAKE, FAKE, ws, nb, None)
    return lib.dcn_cross_attention(r, q, k, v, None, out, lse, ws, nb, None)


def workspace(lib, d, backward):
    n = ctypes.c_size_t(12345)
    f = lib.dcn_cross_attention_backward_workspace_bytes if backward else lib.dcn_cross_attention_workspace_bytes
    return f(ctypes.byref(d), ctypes.byref(n)), n.value


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(query_len=-1), dict(key_len=-1), dict(query_heads=0), dict(key_heads=0), dict(head_dim=0),
    dict(key_heads=3), dict(query_heads=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(q_stride=(-1, 256, 32)), dict(k_stride=(0, -1, 32)), dict(v_stride=(0, 0, -32)),
    dict(mask_stride=-1)], ids=str)
def test_invalid_descriptors(lib, bad, backward):
    d = desc(**bad)
    assert workspace(lib, d, backward) == (dcn.E_ARG, 12345)
    assert status(lib, d, backward) == dcn.E_ARG


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad", [
    dict(dtype=7), dict(head_dim=129), dict(query_len=1 << 31), dict(key_len=1 << 31), dict(batch=1 << 32),
    dict(batch=1 << 20, query_len=1 << 12), dict(batch=1 << 20, key_len=1 << 12)], ids=str)
def test_unsupported_descriptors(lib, bad, backward):
    d = desc(**bad)
    assert workspace(lib, d, backward) == (dcn.E_UNSUPPORTED, 12345)
    assert status(lib, d, backward) == dcn.E_UNSUPPORTED


def test_null_pointers_and_workspace(lib):
    d = desc()
    for n in ("q", "k", "v", "out"):
        assert status(lib, d, False, **{n: None}) == dcn.E_ARG, n
    for n in ("q", "k", "v", "out", "lse", "go"):
        assert status(lib, d, True, **{n: None}) == dcn.E_ARG, n
    assert status(lib, None, False) == dcn.E_ARG and status(lib, None, True) == dcn.E_ARG
    for backward in (False, True):
        f = lib.dcn_cross_attention_backward_workspace_bytes if backward else lib.dcn_cross_attention_workspace_bytes
        assert f(ctypes.byref(d), None) == dcn.E_ARG
        rc, nb = workspace(lib, d, backward)
        assert rc == dcn.OK and workspace(lib, d, backward) == (dcn.OK, nb)
        if nb:
            assert status(lib, d, backward, ws=None, nb=nb) == dcn.E_WORKSPACE
            assert status(lib, d, backward, nb=nb - 1) == dcn.E_WORKSPACE
            assert status(lib, d, backward, ws=WS + 16, nb=nb) == dcn.E_WORKSPACE
    # the row values (8 bytes a row) at least
    assert workspace(lib, d, True)[1] >= 2 * 8 * 300 * 8
    # one token over a long cache is split over workgroups: their parts need room
    assert workspace(lib, desc(batch=1, query_len=1, key_len=16800), False)[1] > 0


def test_nothing_to_do(lib):
    for d in (desc(batch=0), desc(query_len=0)):
        assert workspace(lib, d, False) == (dcn.OK, 0)
        assert lib.dcn_cross_attention(ctypes.byref(d), None, None, None, None, None, None, None, 0, None) == dcn.OK
    d = desc(batch=0)
    assert workspace(lib, d, True) == (dcn.OK, 0)
    assert lib.dcn_cross_attention_backward(ctypes.byref(d), *[None] * 11, 0, None) == dcn.OK


def test_binding_refuses_what_is_not_on_a_gpu(lib):
    import torch
    q, k = torch.zeros(1, 2, 2, 8), torch.zeros(1, 3, 2, 8)
    with pytest.raises(ValueError):
        dcn.cross_attention(q, k, k)
    with pytest.raises(TypeError):
        dcn.cross_attention(q.half(), k.half(), k.half())
