"""Checks on the generated gfx950 code of the operators of a block's attention half, without
a GPU: M0 only feeds the kernels' own LDS loads, and no kernel keeps data in scratch memory
(a spilled register of the attention kernels' sums is a store and a load for every block of keys)."""
import re

import pytest

from tests.test_block_codegen_host import _scratch
from tests.test_codegen_host import _compile_asm, _kernels


@pytest.mark.parametrize("src,kernels,number", [
    ("int8_linear.hip", {"int8_gemm_kernel": 18, "int8_rows_kernel": 15, "int8_reduce_kernel": 3}, 36),
    ("attention.hip", {"attention_small_kernel": 3, "attention_large_kernel": 3, "attention_join_kernel": 6}, 12),
    ("qk_rope.hip", {"qk_rope_kernel": 12}, 12),
])
def test_m0_and_scratch(tmp_path_factory, src, kernels, number):
    text = _compile_asm(tmp_path_factory, src)
    sizes = _scratch(text)
    assert len(sizes) == number
    assert not any(sizes.values()), {k: v for k, v in sizes.items() if v}
    for kernel, count in kernels.items():
        for name, body in _kernels(text, kernel, count).items():
            lines = [ln.strip() for ln in body.splitlines() if ln.strip() and not ln.strip().startswith(";")]
            for i, ln in enumerate(lines):
                if re.search(r"\bm0\b", ln):
                    assert ln.startswith("s_mov_b32 m0, s"), (name, ln)
                    assert lines[i + 1].startswith("global_load_lds"), (name, ln, lines[i + 1])
                elif ln.startswith("global_load_lds"):
                    assert lines[i - 1].startswith("s_mov_b32 m0, s"), (name, lines[i - 1], ln)
