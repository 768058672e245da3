"""scale and eps are read anew in each call: a tensor or array of one value that a program changes
in place (a learned temperature) must not be remembered by its identity.  No GPU: stand-ins with
a tensor's shape, type, device and strides go through the binding's checks, and the descriptors
that a call would pass are compared."""

import ctypes
import os

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn


class OnGpu:
    """What the checks of a call look at."""

    def __init__(self, *shape, dtype=torch.float32):
        like = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self.device, self.stride = like.shape, dtype, torch.device("cuda", 0), like.stride
        self.is_contiguous = like.is_contiguous


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(dcn.LIB_PATH):
        from deformable_convolution_vision_amd import build
        build.build()
    return dcn.load_library()


HOLDERS = {"tensor": lambda v: torch.tensor(v), "array": lambda v: np.array(v, np.float32),
           "one element": lambda v: torch.tensor([v])}


def descriptor(plan, kind):
    return ctypes.cast(plan[0], ctypes.POINTER(kind)).contents


@pytest.mark.parametrize("holder", list(HOLDERS))
def test_a_scale_changed_in_place(holder):
    q, k, scale = OnGpu(1, 3, 4, 32), OnGpu(1, 5, 2, 32), HOLDERS[holder](0.5)
    for value in (0.5, 2.0, 0.25):
        scale[...] = value
        got = descriptor(dcn._attention_plan(*dcn._attention_key(q, k, k, None, scale)), dcn.AttnDesc)
        assert got.scale == value and dcn.attention_desc(q, k, k, scale=scale).scale == value
    # the default is that of the head size
    assert dcn.attention_desc(q, k, k).scale == np.float32(32 ** -0.5)


@pytest.mark.parametrize("holder", list(HOLDERS))
def test_an_eps_changed_in_place(holder):
    x, eps = OnGpu(2, 6, 16), HOLDERS[holder](0.5)
    for value in (0.5, 2.0, 0.25):
        eps[...] = value
        got = descriptor(dcn._norm_plan(*dcn._norm_key(x, 4, None, None, eps, "relu")), dcn.NormDesc)
        assert got.eps == value and dcn.norm_desc(x, 4, eps=eps).eps == value


def test_what_is_no_number_is_refused():
    q, k = OnGpu(1, 3, 4, 32), OnGpu(1, 5, 2, 32)
    for bad in (torch.ones(2), "half", [1.0]):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            dcn.attention_desc(q, k, k, scale=bad)
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            dcn.norm_desc(OnGpu(2, 6, 16), 4, eps=bad)


@pytest.mark.gpu
def test_results_follow_a_changed_scale_and_eps():
    g = torch.Generator().manual_seed(2)
    q, k, v, dout = (torch.randn((2, n, 4, 32), generator=g).cuda() for n in (5, 9, 9, 5))
    scale = torch.tensor(0.5)
    for value in (0.5, 2.0):
        scale.fill_(value)
        out, lse = dcn.cross_attention(q, k, v, scale=scale, return_lse=True)
        want, want_lse = dcn.cross_attention(q, k, v, scale=value, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        for x, y in zip(dcn.cross_attention_backward(dout, q, k, v, out, lse, scale=scale),
                        dcn.cross_attention_backward(dout, q, k, v, out, lse, scale=value)):
            assert torch.equal(x, y)
    eps = torch.tensor(0.5)
    for value in (0.5, 2.0):
        eps.fill_(value)
        assert torch.equal(dcn.group_norm_act(q, 4, eps=eps), dcn.group_norm_act(q, 4, eps=value))
