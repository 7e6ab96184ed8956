"""The division of the work of attention over a cache of 8-bit values and of
calls with trees, run on the CPU with a trap on signed overflow
(tests/attn_work_more_host.cpp)."""
import os
import random
import shutil
import subprocess

import pytest

from test_attn_work import CUDA, HERE, MIXED

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")


@pytest.fixture(scope="module")
def divide(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("attn_work_more") / "attn_work_more_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow,shift,bounds",
                    "-fsanitize-undefined-trap-on-error", "-isystem", CUDA, "-I", os.path.join(HERE, "..", "moe_decode_gb300", "csrc"),
                    os.path.join(HERE, "attn_work_more_host.cpp"), "-o", exe], check=True)

    def run(lens, page=16, window=0, kv_heads=2, group=4, ctas=152):
        width = max(1, max(-(-s // page) for s, _ in lens))
        r = subprocess.run([exe] + [str(v) for v in (page, window, width, kv_heads, group, ctas)] + [f"{s},{n}" for s, n in lens],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, (r.returncode, r.stdout, lens, page, window, kv_heads, group, ctas)

    return run


@pytest.mark.parametrize("lens", MIXED, ids=lambda v: "-".join("%d,%d" % p for p in v[:4]))
@pytest.mark.parametrize("window", [0, 1, 128, (1 << 31) - 1])
def test_every_tile_once(divide, lens, window):
    for group, ctas, page in ((1, 152, 16), (4, 1, 48), (7, 61, 16), (16, 256, 112), (32, 152, 1024)):
        divide(lens, page=page, window=window, group=group, ctas=ctas)


def test_every_tile_once_at_random(divide):
    rng = random.Random(11)
    for _ in range(40):
        lens = [(int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 8)) - 1) for _ in range(rng.randint(1, 40))]
        divide(lens, page=rng.choice([16, 32, 48, 64, 128]), window=rng.choice([0, 0, rng.randint(1, 4000)]),
               kv_heads=rng.choice([1, 2, 8]), group=rng.choice([1, 3, 4, 7, 16, 32]), ctas=rng.choice([1, 7, 61, 152]))


@pytest.mark.parametrize("new", [1, 20, 300])
def test_up_to_the_last_position(divide, new):
    for page in (16, 1024):
        for short in (0, 33, 128):
            seq = (1 << 31) - 1 - short
            divide([(seq, new), (seq - 1, 1)], page=page, window=500, ctas=61)
