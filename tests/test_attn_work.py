"""The division of the paged attention's work over the CTAs (the part of the
kernels that is integer arithmetic alone), run on the CPU with a trap on signed
overflow: tests/attn_work_host.cpp says what is checked."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")


@pytest.fixture(scope="module")
def divide(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("attn_work") / "attn_work_host")
    # (the trap needs no run-time library of the sanitizer)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow,shift,bounds",
                    "-fsanitize-undefined-trap-on-error", "-isystem", CUDA, "-I", os.path.join(HERE, "..", "moe_decode_gb300", "csrc"),
                    os.path.join(HERE, "attn_work_host.cpp"), "-o", exe], check=True)

    def run(lens, page=16, window=0, width=None, kv_heads=2, group=4, ctas=152):
        width = width or max(1, max(-(-s // page) for s, _ in lens))
        r = subprocess.run([exe] + [str(v) for v in (page, window, width, kv_heads, group, ctas)] + [f"{s},{n}" for s, n in lens],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, (r.returncode, r.stdout, lens, page, window, width, kv_heads, group, ctas)

    return run


MIXED = [[(1, 1)], [(128, 1), (129, 1), (127, 2), (256, 128)], [(900, 200), (1, 1), (0, 0), (333, 5), (2049, 1)],
         [(3, 7), (0, 2), (0, 0), (150, 160), (64, 1)], [(16383, 8192), (100, 1)], [(700, 40)] * 65]


@pytest.mark.parametrize("lens", MIXED, ids=lambda v: "-".join("%d,%d" % p for p in v[:4]))
@pytest.mark.parametrize("window", [0, 1, 128, 1000])
def test_every_tile_once(divide, lens, window):
    for group, ctas, page in ((1, 152, 16), (4, 1, 48), (7, 61, 8), (16, 256, 136), (32, 152, 1024)):
        divide(lens, page=page, window=window, group=group, ctas=ctas)


def test_every_tile_once_at_random(divide):
    rng = random.Random(7)
    for _ in range(60):
        lens = [(int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 10)) - 1) for _ in range(rng.randint(1, 40))]
        divide(lens, page=rng.choice([8, 16, 24, 48, 64, 128, 136]), window=rng.choice([0, 0, rng.randint(1, 4000)]),
               kv_heads=rng.choice([1, 2, 8]), group=rng.choice([1, 3, 4, 7, 16, 32]), ctas=rng.choice([1, 7, 61, 152]))


@pytest.mark.parametrize("lens", MIXED, ids=lambda v: "-".join("%d,%d" % p for p in v[:4]))
@pytest.mark.parametrize("window", [1 << 28, 1 << 30, (1 << 31) - 3, (1 << 31) - 2, (1 << 31) - 1])
def test_windows_wider_than_everything(divide, lens, window):
    """Next to rows at negative positions too."""
    for group, ctas in ((1, 152), (4, 3), (16, 152)):
        divide(lens, window=window, group=group, ctas=ctas)


@pytest.mark.parametrize("new", [1, 6, 20, 300])
@pytest.mark.parametrize("page", [8, 136, 1024])
@pytest.mark.parametrize("window", [1, 500, 5000])
def test_up_to_the_last_position(divide, new, page, window):
    """Keys up to 2^31 - 2: their numbers rounded up to whole tiles do not fit 32
    bits."""
    for short in (0, 1, 33, 127, 128, 1000):
        seq = (1 << 31) - 1 - short
        divide([(seq, new), (seq - 1, 1)], page=page, window=window, width=-(-seq // page), ctas=61)
