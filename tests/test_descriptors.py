"""The descriptors that the binding gives out for the raw entry points are the caller's own: altering one does
not reach what later calls of the same sizes pass to the library."""

import ctypes

import pytest
import torch

import deformable_convolution_vision_amd as dcn


class OnGpu:
    """What the checks look at in a tensor on a GPU, on a host that has none."""

    def __init__(self, shape, dtype=torch.float32):
        t = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self.device, self._strides = t.shape, dtype, torch.device("cuda:0"), t.stride()

    def stride(self):
        return self._strides


def ints(*shape):
    return OnGpu(shape, torch.int32)


def rotary():
    return dcn.rotary_desc(OnGpu((2, 5, 3, 16)), OnGpu((2, 5, 1)), OnGpu((8,)), (8,))


def residual():
    x = OnGpu((2, 5, 64))
    return dcn.residual_desc(x, x, scale=OnGpu((64,)))


def append():
    k, pages = OnGpu((2, 5, 3, 16)), OnGpu((7, 4, 3, 16))
    return dcn.append_desc(k, k, pages, pages, ints(2, 3), ints(2), frequencies=OnGpu((8,)), sections=(8,))


def paged():
    pages = OnGpu((7, 4, 3, 16))
    return dcn.paged_desc(OnGpu((2, 6, 16)), pages, pages, ints(2, 3), ints(2))


PLANS = {rotary: dcn._rotary_plan, residual: dcn._residual_plan, append: dcn._append_plan, paged: dcn._paged_plan}


@pytest.mark.parametrize("make", list(PLANS), ids=lambda f: f.__name__)
def test_a_descriptor_is_the_callers_own(make):
    PLANS[make].cache_clear()
    first = make()
    assert PLANS[make].cache_info().currsize == 1        # a plan of these sizes is kept now
    was = bytes(first)
    ctypes.memset(ctypes.addressof(first), 0x7f, ctypes.sizeof(first))
    second = make()
    assert PLANS[make].cache_info().hits == 1            # and was used again
    assert second is not first and type(second) is type(first) and bytes(second) == was


@pytest.mark.gpu
def test_calls_after_a_descriptor_was_altered():
    g = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g).cuda()

    x, freq, pages = normal(2, 5, 3, 16), torch.rand(8, generator=g).cuda(), normal(7, 4, 3, 16)
    at = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5, 1)
    table, starts = torch.tensor([[1, 4, 5], [2, 0, 6]], dtype=torch.int32, device="cuda"), at[:, 0, 0].contiguous()
    stream, branch, q = normal(2, 5, 64), normal(2, 5, 64), normal(2, 6, 16)

    def calls():
        kp, vp = pages.clone(), pages.clone()
        n = dcn.paged_append(x, x, kp, vp, table, starts, frequencies=freq, sections=(8,))
        return [dcn.rotary_positions(x, at, freq, (8,)), *dcn.residual_norm(stream, branch), kp, vp, n,
                dcn.paged_attention(q, kp, vp, table, n)]

    want = calls()
    # (each to a smaller problem, so that a call that it reached would leave results out)
    dcn.rotary_desc(x, at, freq, (8,)).length = 2
    dcn.residual_desc(stream, branch).positions = 2
    dcn.append_desc(x, x, pages, pages, table, starts, frequencies=freq, sections=(8,)).length = 2
    dcn.paged_desc(q, pages, pages, table, starts).batch = 1
    assert all(torch.equal(a, b) for a, b in zip(calls(), want))
