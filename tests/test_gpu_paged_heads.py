"""dcn_paged_attention with more than 16 query heads on a key head (several tiles of its 16 rows) over caches
that are divided into parts, within the bounds of fp32 weights."""

import pytest
import torch

import deformable_convolution_vision_amd as dcn
import test_gpu_paged
from test_gpu_paged_weights import compare

pytestmark = pytest.mark.gpu

# name: lengths, Hq, Hkv, D, page size
CASES = {
    "40_on_2": ([5000, 3, 1700], 40, 2, 64, 16),
    "40_on_2_wide": ([5000, 3, 1700], 40, 2, 128, 16),
    "17_on_1": ([2900, 0, 65], 17, 1, 128, 64),
    "33_on_1": ([3100, 700], 33, 1, 32, 7),
    "48_on_1_odd": ([4000], 48, 1, 45, 32),
    "34_on_2_narrow_rounds": ([300 + (97 * i) % 2000 for i in range(40)], 34, 2, 64, 32),
    "lists_40_on_2": ([(131 * i) % 60 for i in range(70)] + [2600, 1900], 40, 2, 64, 32),
    "lists_40_on_2_wide": ([(131 * i) % 60 for i in range(70)] + [2600, 1900], 40, 2, 128, 16),
    "lists_17_on_1": ([(17 * i) % 90 for i in range(65)] + [1700, 0, 1800], 17, 1, 37, 24),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_tiles_in_parts(name, dtype, monkeypatch):
    print(f"[gpu-test] paged heads {name} {dtype}", flush=True)
    monkeypatch.setitem(test_gpu_paged.ATTENTION, name, CASES[name])
    args = test_gpu_paged.make(name, dtype)
    assert dcn.dcn_paged_attention_workspace_bytes(dcn.paged_desc(*args)) > 0, "the case is not divided into parts"
    compare(args, dtype, name, CASES[name][3] ** -0.5)
    out = dcn.paged_attention(*args)
    assert torch.equal(out, dcn.paged_attention(*args)), "the same call gave other bits"
    # every query head on its own, over its key head: nothing of another tile's parts
    q, k, v, table, lengths = args
    g = q.shape[1] // k.shape[2]
    for h in (0, 15, 16, g - 1, q.shape[1] - 1):
        only = [t[:, :, h // g:h // g + 1] for t in (k, v)]
        alone = dcn.paged_attention(q[:, h:h + 1], *only, table, lengths)
        # (its workgroups divide the sequences otherwise: twice the bound of one, in which bf16's 3n products make
        # sqrt(3) of acc(n), and two roundings)
        ref = test_gpu_paged.reference(q[:, h:h + 1], *only, table, lengths, "f32")
        step = 0.0 if dtype == "f32" else torch.finfo(torch.bfloat16).eps
        off = (alone[:, 0].double() - out[:, h].double()).abs().cpu().numpy()
        assert (off <= 4 * ref[1][:, 0] + 1.01 * step * abs(ref[0][:, 0])).all(), h
