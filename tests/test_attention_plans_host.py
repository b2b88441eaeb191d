"""Which kernels the GPU tests of a block's attention half reach: their sizes put to the planners of
csrc/attention.hip and csrc/int8_linear.hip (tests/host/plan_driver.cpp, on the CPU).  A
change of the planners that moves a size to another kernel shows here, and not as a kernel
that no test runs."""
import os
import subprocess

import pytest

pytest.importorskip("torch")
from tests import test_gpu_attention_large as L  # noqa: E402
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


def _attention_sizes(lengths, shape, split, window, sinks):
    """T, B, group, n_kv, D, the table's keys, window and sinks of test_gpu_attention_large.case."""
    D, n_q, n_kv, page = shape
    rows, keys = L.form(D, split)
    pages = max(1, keys // page, *(-(-kv // page) for _, kv in lengths))
    return max(sum(n for n, _ in lengths), -(-rows // n_q)), len(lengths), n_q // n_kv, n_kv, D, pages * page, window, sinks


def test_attention_calls_take_the_kernel_for_many_rows(plans):
    calls = list(L.calls())
    got = plans("attention", [_attention_sizes(*c[:5]) for c in calls])
    reached = set()
    for call, (small, large, small_rows, _, large_splits) in zip(calls, got):
        assert large and (large_splits > 1) == call[5], (call, large, large_splits)
        assert small == (len(call[0]) > 1) and small_rows == (64 if small else 0)  # which rows the other kernel takes
        reached.add((call[1][0], small, min(large_splits, 3)))
    assert reached == {(D, small, splits) for D in (64, 128, 256) for small in (0, 1) for splits in (1, 2, 3)}


def test_sizes_of_the_calls(plans):
    """_attention_sizes gives what the cases hold."""
    for lengths, shape, split in ((L.BESIDE[0], L.SHAPES[1], False), (L.LONG[1], L.SHAPES[4], True), (L.EMPTY, L.ONE[64], False)):
        try:
            made = {}
            keep, L.S._case = L.S._case, lambda *a, **kw: made.update(a=a, kw=kw)
            L.case(0, lengths, shape, split)
        finally:
            L.S._case = keep
        page, need = made["a"][5], max([-(-kv // made["a"][5]) for _, kv in lengths] + [1])
        T, _, _, _, _, keys, _, _ = _attention_sizes(lengths, shape, split, 0, 0)
        assert (sum(n for n, _ in lengths) + made["kw"]["spare_rows"], (need + made["kw"]["wide"]) * page) == (T, keys)


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


def test_splits_of_few_rows_fill_the_device_and_no_more(plans):
    """Workgroups of the kernel for few rows: tiles of 16 rows (a token has several where more than 16 query heads
    share a key head) times splits are at most 12, 8 or 4 a CU, by head size, or there are no splits."""
    import random
    rng = random.Random(1)
    sizes = []
    for _ in range(20000):
        n_kv = 2 ** rng.randrange(0, 5)
        sizes.append((int(2 ** rng.uniform(0, 9)), int(2 ** rng.uniform(0, 7)), int(2 ** rng.uniform(0, 10)) // n_kv or 1, n_kv,
                      rng.choice([64, 128, 256]), 16 * int(2 ** rng.uniform(0, 12)), 0, 0))
    split = 0
    for size, (small, _, _, splits, _) in zip(sizes, plans("attention", sizes)):
        T, _, group, n_kv, D = size[:5]
        if small and splits > 1:
            split += 1
            assert splits * (T * group // 16) * n_kv <= {64: 12, 128: 8, 256: 4}[D] * 256, (size, splits)
    assert split > 2000
