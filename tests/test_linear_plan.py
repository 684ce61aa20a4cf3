"""What a matrix product may read and how it is cut into tiles, without a GPU: the
arithmetic of csrc/linear_plan.h, compiled for the host."""
import ctypes
import os
import random
import subprocess

import pytest

from linear_tiles import TILES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include "linear_plan.h"
extern "C" int scale_span(int rows, int stride, int blocks) { return st::scale_span(rows, stride, blocks); }
extern "C" void choose(long long m, long long n, long long k, int type, int widened, int cols, long long* out) {
  const st::Choice c = st::choose(m, n, k, type, widened != 0, cols != 0);
  out[0] = c.shape; out[1] = c.splits; out[2] = c.per_split;
  const st::Shape h = c.shape == st::kFewShape ? st::Shape{32, st::kFewRows, 1} : st::shape_of(type, c.shape);
  out[3] = h.ta; out[4] = h.tb; out[5] = h.per_cu; out[6] = st::stage_steps(type);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("linear_plan")
    (d / "plan.cpp").write_text(SOURCE)
    out = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "halo_sharded_conv_amd", "csrc"),
                    "-I", os.path.join(ROOT, "include"), str(d / "plan.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.mark.parametrize("rows", [1, 2, 33, 256])
@pytest.mark.parametrize("blocks", [1, 3, 4, 5, 7, 8, 9, 32, 33])
@pytest.mark.parametrize("before", [0, 4, 16, 64])
def test_scale_bytes_end_with_the_last_row(plan, rows, blocks, before):
    """Scales as the last columns of a buffer `before` bytes wider: what is read, 16
    bytes of every row at a time, word by word while it starts inside the span, holds
    every block's byte and no word behind the buffer's last row."""
    words = -(-blocks // 4) * 4
    stride = before + words
    span = plan.scale_span(rows, stride, blocks)
    read = {r * stride + at + w for r in range(rows) for at in range(0, words, 16) for w in (0, 4, 8, 12) if r * stride + at + w < span}
    assert {r * stride + w for r in range(rows) for w in range(0, words, 4)} <= read
    assert max(read) + 4 <= rows * stride - before


TYPES = {"f32": 0, "bf16": 1, "mx8": 2}


def choose(plan, m, n, k, dtype, widened=False, cols=False):
    """(shape, splits, stages a split, tile, tiles a compute unit, steps a stage)"""
    out = (ctypes.c_longlong * 7)()
    q = ctypes.c_longlong
    plan.choose(q(m), q(n), q(k), TYPES[dtype], int(widened), int(cols), out)
    return out[0], out[1], out[2], (out[3], out[4]), out[5], out[6]


def product_sizes(product, rows, cin, cout):
    """(rows, channels, contraction) of one product of st_linear or st_linear_backward."""
    return {"y": (rows, cout, cin), "dx": (rows, cin, cout), "dw": (cout, cin, rows)}[product]


@pytest.mark.parametrize("product,dtype,rows,cin,cout,widened,tile,stages", TILES)
def test_tiles_of_the_sizes(plan, product, dtype, rows, cin, cout, widened, tile, stages):
    m, n, k = product_sizes(product, rows, cin, cout)
    _, splits, per, got, per_cu, steps = choose(plan, m, n, k, dtype, widened, product != "y")
    assert got == tile
    assert stages == (per if splits > 1 else -(-k // steps))
    tiles = -(-n // tile[0]) * -(-m // tile[1]) * splits
    assert tiles > 256 * per_cu                            # more than one a workgroup


def test_every_tile_has_its_sizes():
    """Every tile of every product and type, by one stage, two, three and more."""
    seen = {}
    for product, dtype, _, _, _, widened, tile, stages in TILES:
        seen.setdefault((product, dtype, widened, tile), set()).add(stages)
    assert set(seen) == {*(("y", d, False, t) for d in ("bf16", "mx8") for t in ((256, 256), (128, 64), (64, 64))), ("y", "mx8", True, (128, 64)),
                         *((p, "bf16", False, t) for p in ("dx", "dw") for t in ((256, 256), (128, 64), (64, 64))),
                         *((p, "f32", False, t) for p in ("y", "dx", "dw") for t in ((128, 128), (128, 64), (64, 64)))}
    for key, stages in seen.items():
        assert key[3] == (128, 128) or len(stages) >= 3, key


def test_large_fp32_tiles_have_split_sums(plan):
    """Which is why they need no other epilogue than the partial sums'."""
    rng = random.Random(1)
    size = lambda lo, hi: int(round(2 ** rng.uniform(lo, hi)))  # noqa: E731
    large = 0
    for _ in range(20000):
        shape, splits = choose(plan, size(0, 20), size(0, 14), size(0, 20), "f32", cols=rng.random() < 0.5)[:2]
        assert shape != 0 or splits > 1
        large += shape == 0
    assert large > 0
