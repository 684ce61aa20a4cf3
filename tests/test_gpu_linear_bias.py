"""The bias of a matrix product: added once, to the whole sum, and rounded once."""
import pytest
import torch

from helpers import say
from linear_tiles import TILES
from test_gpu_linear_tiles import blank, held, numbers, same

pytestmark = pytest.mark.gpu

SIZES = [(m, k, n, dtype) for product, dtype, m, k, n, *_ in TILES if product == "y"]
FEW = [(m, k, n, dtype) for dtype in ("bf16", "f32", "mx8") for m, k, n in
       ((1, 1, 8), (5, 11, 520), (33, 1000, 257), (64, 8192, 96), (70, 1, 40), (150, 11, 200), (300, 9000, 260), (5092, 11, 3264))]


@pytest.mark.parametrize("m,k,n,dtype", FEW + SIZES)
def test_bias_is_rounded_once(gpu_lib, m, k, n, dtype):
    """Products of whole numbers have exact sums (below 2^24); a bias of 24 bits added to
    one is off by the rounding of the result and by nothing else: the bits of the
    64-bit sum in fp32 (which holds it exactly: whole numbers below 2^24 and a bias
    of at least 2^-26 or zero need 50 bits), and of its codes in 8 bits."""
    say(f"linear {m}x{k}x{n} {dtype}: bias")
    draw = numbers(m + k + n)
    xf, wf = draw(m, k), draw(n, k)
    gen = torch.Generator(device="cuda").manual_seed(n)
    b = torch.randn(n, generator=gen, device="cuda")
    b[b.abs() < 2.0 ** -3] = 0.0                          # (so that the lowest bit is 2^-26 or higher)
    x, w = held(gpu_lib, xf, dtype), held(gpu_lib, wf, dtype)
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, dtype)), dtype=torch.uint8, device="cuda")
    z = (xf.double() @ wf.double().t() + b.double()).float()
    # 8-bit operands with nothing but bf16 outputs take the other products: exact here too
    for y, pre, act in (("f32", "", "none"), ("f32", "mx8", "relu"), ("bf16", "", "none"), ("bf16", "bf16", "relu")):
        yo, po = blank(gpu_lib, y, m, n), blank(gpu_lib, pre, m, n) if pre else (None, None)
        gpu_lib.st_linear(x, w, b, yo[0], act=act, pre=po[0], workspace=ws)
        assert same(gpu_lib, yo, torch.relu(z) if act == "relu" else z, y), f"y {y} {act}"
        assert not pre or same(gpu_lib, po, z, pre), f"pre {pre}"
