"""What a matrix product may read and how it is cut into tiles, without a GPU: the
arithmetic of csrc/linear_plan.h, compiled for the host."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include "linear_plan.h"
extern "C" int scale_span(int rows, int stride, int blocks) { return st::scale_span(rows, stride, blocks); }
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
