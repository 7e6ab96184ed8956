"""Where the attention's padding rows begin, run on the CPU
(tests/attn_padding_host.cpp)."""
import os
import shutil
import subprocess

import pytest

from test_attn_work import CUDA, HERE

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")


@pytest.fixture(scope="module")
def padding(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("attn_padding") / "attn_padding_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow,shift,bounds",
                    "-fsanitize-undefined-trap-on-error", "-isystem", CUDA, "-I", os.path.join(HERE, "..", "moe_decode_gb300", "csrc"),
                    os.path.join(HERE, "attn_padding_host.cpp"), "-o", exe], check=True)

    def run(T, q_start):
        return int(subprocess.run([exe] + [str(v) for v in [T] + q_start], capture_output=True, text=True, timeout=60, check=True).stdout)

    return run


@pytest.mark.parametrize("T,q_start,first", [
    (4, [0, 2, 3], 3), (4, [0, 0], 0), (4, [0, 4], 4), (5, [0, 3, 3, 3], 3), (7, [-1, 2, 3], 3), (7, [0, -3, 2], 2),
    # the last request ends beyond the rows, or before it begins
    (4, [0, 2, 900], 4), (4, [0, 2, (1 << 31) - 1], 4), (4, [0, 2, -1], 4), (4, [0, 3, 2], 4), (4, [0, 9, 3], 4), (4, [0, -1], 4),
    (4, [0, -2, -1], 4), (4, [0, -(1 << 31)], 4), (4, [0, (1 << 31) - 1, -(1 << 31)], 4)])
def test_padding(padding, T, q_start, first):
    assert padding(T, q_start) == first
