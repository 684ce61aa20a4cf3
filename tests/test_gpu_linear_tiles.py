"""Matrix products in every tile that there is, over several tiles a workgroup, and
their 8-bit operands and outputs bit for bit."""
import math

import numpy as np
import pytest
import torch

from helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", [(5, 40), (40, 130), (300, 200), (1100, 600)])
@pytest.mark.parametrize("k", [40, 128, 200, 1000, 4104])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_scales_that_end_a_buffer(gpu_lib, m, n, k, y):
    """Scales as the last columns of a wider buffer, whose last byte is theirs: the
    bits of scales that lie by themselves."""
    say(f"linear {m}x{k}x{n} mx8, y {y}, scales in the last columns of a buffer")
    rng = np.random.default_rng(m + n + k)
    own, ends = [], []
    for rows, size in ((m, 1.0), (n, 1 / math.sqrt(k))):
        o = gpu_lib.mx8_empty(rows, k)
        o.scales.zero_()
        gpu_lib.st_mx8_store(torch.from_numpy(np.float32(size * rng.normal(size=(rows, k)))).cuda(), o)
        words = o.scales.shape[1]
        wide = torch.full((rows, 16 + words), 0xFF, dtype=torch.uint8, device="cuda")
        wide[:, 16:] = o.scales
        own.append(o)
        ends.append(gpu_lib.Mx8(o.codes, wide[:, 16:], k))
    got = []
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, "mx8")), dtype=torch.uint8, device="cuda")
    for x, w in (own, ends):
        out = torch.full((m, n), math.nan, device="cuda").to(torch.float32 if y == "f32" else torch.bfloat16)
        gpu_lib.st_linear(x, w, None, out, workspace=ws)
        got.append(out)
    assert bool(torch.isfinite(got[0]).all()) and torch.equal(*got)
