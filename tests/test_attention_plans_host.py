"""Which kernels the GPU tests of a block's attention half reach: their sizes put to the planners of
csrc/attention.hip and csrc/int8_linear.hip (tests/host/plan_driver.cpp, on the CPU).  A
change of the planners that moves a size to another kernel shows here, and not as a kernel
that no test runs."""
import os
import subprocess

import pytest

pytest.importorskip("torch")
from tests import test_gpu_int8_tiles as I  # noqa: E402
from tests.test_host_sanitized import CSRC, ROOT, _hipcc  # noqa: E402

DRIVER = os.path.join(ROOT, "tests", "host", "plan_driver.cpp")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """The plans of a list of sizes, by source."""
    if not os.path.exists(_hipcc()):
        pytest.skip("hipcc not available")
    made = {}

    def ask(source, sizes):
        if source not in made:
            made[source] = str(tmp_path_factory.mktemp("plan") / "driver")
            cmd = [_hipcc(), "-x", "hip", "--cuda-host-only", "--offload-arch=gfx950", "-std=c++17", "-O1", "-ffp-contract=off",
                   f'-DPLANNER="{source}.hip"', f"-D{source.upper()}", "-I", os.path.join(ROOT, "include"), "-I", CSRC, DRIVER, "-o", made[source]]
            res = subprocess.run(cmd, capture_output=True, text=True)
            assert res.returncode == 0, res.stderr[-3000:]
        res = subprocess.run([made[source]], input="".join(" ".join(map(str, s)) + "\n" for s in sizes), capture_output=True, text=True, timeout=60)
        assert res.returncode == 0
        out = [tuple(map(int, ln.split())) for ln in res.stdout.splitlines()]
        assert len(out) == len(sizes)
        return out
    return ask


def test_int8_sizes_take_the_kernel_they_name(plans):
    sizes = [(s, key) for table in (I.TILED, I.ROWS) for key, list_ in table.items() for s in list_]
    got = plans("int8_linear", [s for s, _ in sizes])
    for (size, key), (rt, mt, tile, splits) in zip(sizes, got):
        assert key == ((rt, mt) if rt else (tile, splits)), size
        assert (size in sum(I.ROWS.values(), [])) == (rt > 0)


def test_int8_plans_that_no_size_here_reaches(plans):
    """Every plan of a wide choice of sizes is one that the tables name."""
    import random
    rng = random.Random(0)
    sizes = [(int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 17)), 16 * int(2 ** rng.uniform(0, 12))) for _ in range(100000)]
    for size, (rt, mt, tile, splits) in zip(sizes, plans("int8_linear", sizes)):
        assert (rt, mt) in I.ROWS if rt else (tile, splits) in I.TILED, (size, tile, splits)
