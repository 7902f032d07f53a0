"""The many-token product in 4 bits reads nothing behind its operands: every load of a
tile of any size is inside its rows and tokens by its own address, whatever a buffer
descriptor's range counts, and every column meets its token once (CPU only: the
addresses' own functions in a small program)."""
import os
import random
import subprocess

import pytest

from test_q4_plans_cpu import CSRC, CXX, HERE

pytestmark = pytest.mark.cpu


def test_loads_of_a_tile(tmp_path):
    if CXX is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "q4_loads")
    subprocess.run([CXX, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "plans", "q4_loads.cpp"), "-o", exe], check=True)
    rng = random.Random(3)
    sizes = [(r, m, i) for r in (1, 15, 16, 17, 63, 64, 65, 240, 241, 255, 256) for m in (1, 15, 16, 17, 48, 49, 63, 64)
             for i in (32, 64, 96, 128, 160, 224, 256, 288, 1056)]
    sizes += [(rng.randint(1, 256), rng.randint(1, 64), 32 * rng.randint(1, 40)) for _ in range(500)]
    out = subprocess.run([exe], input="".join("%d %d %d\n" % s for s in sizes), capture_output=True, text=True,
                         check=True, timeout=120).stdout.splitlines()
    assert len(out) == len(sizes)
    for s, line in zip(sizes, out):
        assert line == "0 0 0 0", (s, line)
