"""The error bound that the headers state for SiLU(g) u = g u / (1 + e^-g) of
ternary_gated_linear, against the kernel's own formula: the fp32 product g (-log2 e)
and constant as they stand in the source, everything after them exact.  What is left
of the bound has to hold the rest: the native exponential and reciprocal (1 ulp each,
two units of 2^-24), the sum and the two products (one each), 7 in all."""
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INTERNAL = os.path.join(ROOT, "ternary_weight_linear_block_amd", "csrc", "twl_internal.h")


def _text(path):
    return " ".join(ln.strip().lstrip("/*").strip() for ln in open(path))


@pytest.mark.parametrize("path", [os.path.join(ROOT, "include", "twl.h"), INTERNAL])
def test_stated_bound_holds(path):
    m = re.search(r"within \((?:([\d.]+) )?\|g\| \+ ([\d.]+)\) 2\^-24\s+relative", _text(path))
    assert m, "no bound stated"
    slope, const = float(m.group(1) or 1), float(m.group(2))
    c = re.search(r"exp2f\(g \* -(0x1\.[0-9a-f]+p\+0)f\)", open(INTERNAL).read())
    log2e = np.float32(float.fromhex(c.group(1)))
    assert abs(float(log2e) * np.log(2) - 1) < 2.0 ** -24
    # every float of some intervals, and a spread over the whole range where 1 + e^-g stays normal
    parts = [np.arange(lo.view(np.int32), hi.view(np.int32), dtype=np.int32).view(np.float32)
             for lo, hi in (np.array(v, np.float32) for v in ((44.0, 44.5), (86.5, 87.0), (11.0, 11.02), (1.0, 1.01)))]
    g = np.concatenate(parts + [np.random.default_rng(0).uniform(0, 87, 10 ** 6).astype(np.float32)])
    for sign in (-1.0, 1.0):
        t = (np.float32(-sign) * (g * log2e)).astype(np.float64)
        exact = 1.0 / (1.0 + np.exp(-sign * g.astype(np.float64)))
        err = np.abs((1.0 / (1.0 + np.exp2(t))) / exact - 1.0) * 2.0 ** 24
        over = err + 7.0 - (slope * g + const)
        at = int(np.argmax(over))
        assert over[at] <= 0, f"g={sign * g[at]!r}: {err[at]:.2f} + 7 units of 2^-24, stated {slope * g[at] + const:.2f}"
