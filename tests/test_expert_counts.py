"""How the experts' products count blocks and steps of rows, up to the most
rows that a call can have: in constant expressions, where the compiler refuses
what overflows.  And a call that no launch can hold."""

import os
import shutil
import subprocess

import pytest
import torch

from combine_ep_layout_04_amd import ep

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_ep_layout_04_amd", "csrc")

SRC = r"""
#include <initializer_list>
#include "ep_count.h"
using namespace ep;
constexpr int kMost = 2147483647;
constexpr bool counts(int n, int size)
{
    return blocks_of(n, size) == (int)(((int64_t)n + size - 1) / size);
}
constexpr bool all_counts()
{
    for (int size : {16, 32, 64, 128, 256})
        for (int k = 0; k <= 2 * size; ++k)
            if (!counts(k, size) || !counts(kMost - k, size)) return false;
    return true;
}
static_assert(all_counts(), "blocks of rows");
static_assert(blocks_of(0, 16) == 0 && blocks_of(-5, 16) == 0 && blocks_of(-kMost - 1, 256) == 0, "none");
constexpr bool all_steps()
{
    for (int n : {1, 63, 64, 65, 128, 1000, kMost - 63, kMost - 1, kMost}) {
        const int last = blocks_of(n, 64) - 1;
        for (int s = last > 3 ? last - 3 : 0; s <= last; ++s)
            if (whole_step(s, n) != ((int64_t)s * 64 + 64 <= n)) return false;
    }
    return true;
}
static_assert(all_steps(), "whole steps");
static_assert(max_row_blocks(kMost, 1024, 16) == kMost / 16 + 1024LL && max_row_blocks(3, 8, 16) == 3, "most");
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a C++ compiler")
def test_counts_of_rows(tmp_path):
    src = tmp_path / "counts.cpp"
    src.write_text(SRC)
    res = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsyntax-only", f"-I{CSRC}", str(src)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake pointers must never reach a launch on a real GPU")
def test_more_threads_than_a_launch_can_have():
    """8-bit gated halves that are not whole blocks of 128 take a workgroup per
    tile: a call of 2^24 tiles is refused before any launch."""
    fake, R = 0x100000, (1 << 31) - 1

    def call(rows):
        return ep.lib().ep_expert_matmul_fp8(fake, 1, 16, 1, fake, 0, 1, 1, fake, fake, fake, 2, 2, 16, 1, fake, None,
                                             rows, fake, 0, 1, None)
    assert call(R) == 2 and "threads" in ep.last_error()
