"""The largest sizes that rotary positions, joins, append and paged attention take, as dcn.h states them, and
one more.  No GPU: a call that passes the descriptor's checks ends at a pointer that is not there."""

import pytest

import deformable_convolution_vision_amd as dcn
from test_decoder_abi import append, lib, paged, residual, rotary, run_append, run_join, run_paged, run_rotary, size  # noqa: F401

MOST = (1 << 31) - 1


@pytest.mark.parametrize("over, taken", [
    (dict(head_dim=128), True), (dict(head_dim=129), False),
    (dict(batch=(1 << 27) - 1, query_heads=1, key_heads=1), True), (dict(batch=1 << 27, query_heads=1, key_heads=1), False),
    (dict(batch=1, query_heads=(1 << 27) - 1, key_heads=1), True), (dict(batch=1, query_heads=1 << 27, key_heads=1), False),
    (dict(num_pages=MOST), True), (dict(num_pages=MOST + 1), False),
    (dict(max_pages=MOST - 65536, page_size=1), True), (dict(max_pages=MOST - 65535, page_size=1), False),
    (dict(max_pages=1, page_size=MOST - 65536), True), (dict(max_pages=1, page_size=MOST - 65535), False),
    (dict(max_pages=MOST, page_size=1), False)], ids=str)
def test_paged_attention(lib, over, taken):  # noqa: F811
    d = paged(**over)
    rc, nb = size(lib.dcn_paged_attention_workspace_bytes, d)
    assert rc == (dcn.OK if taken else dcn.E_UNSUPPORTED) and (nb > 12345 if taken else nb == 12345)
    assert run_paged(lib, d, q=None) == (dcn.E_ARG if taken else dcn.E_UNSUPPORTED)


@pytest.mark.parametrize("over, taken", [
    (dict(head_dim=512), True), (dict(head_dim=513), False),
    (dict(max_pages=MOST, page_size=1), True), (dict(max_pages=MOST + 1, page_size=1), False),
    (dict(max_pages=1, page_size=MOST), True), (dict(max_pages=1, page_size=MOST + 1), False),
    (dict(num_pages=MOST), True), (dict(num_pages=MOST + 1), False),
    # 8 + 2 + 2 heads
    (dict(batch=1, length=MOST // 12), True), (dict(batch=1, length=MOST // 12 + 1), False),
    (dict(batch=MOST // 12, length=0), True), (dict(batch=MOST // 12 + 1, length=0), False)], ids=str)
def test_append(lib, over, taken):  # noqa: F811
    assert run_append(lib, append(**over), starts=None) == (dcn.E_ARG if taken else dcn.E_UNSUPPORTED)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("over, taken", [
    (dict(head_dim=512), True), (dict(head_dim=513), False),
    (dict(batch=1, length=MOST // 8), True), (dict(batch=1, length=MOST // 8 + 1), False),
    (dict(batch=1, length=1, heads=MOST), True), (dict(batch=1, length=1, heads=MOST + 1), False)], ids=str)
def test_rotary(lib, over, taken, backward):  # noqa: F811
    assert run_rotary(lib, rotary(**over), backward, freq=None) == (dcn.E_ARG if taken else dcn.E_UNSUPPORTED)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("over, taken", [
    (dict(channels=8192), True), (dict(channels=8193), False),
    (dict(batch=1, positions=MOST), True), (dict(batch=1, positions=MOST + 1), False),
    (dict(batch=65530), True), (dict(batch=65531), False),
    (dict(batch=MOST, positions=1, gate=0), True), (dict(batch=MOST + 1, positions=1, gate=0), False)], ids=str)
def test_join(lib, over, taken, backward):  # noqa: F811
    d = residual(**over)
    assert size(lib.dcn_residual_norm_backward_workspace_bytes, d)[0] == (dcn.OK if taken else dcn.E_UNSUPPORTED)
    assert run_join(lib, d, backward, x=None) == (dcn.E_ARG if taken else dcn.E_UNSUPPORTED)
