"""Checks on the generated gfx950 code of the block operators, without a GPU: the
gated decode kernels keep M0 to their own LDS loads (as the linear layer's do, see
test_codegen_host.py), and no kernel of the usual sizes keeps data in scratch
memory (an array that the compiler left there made the adapter kernels three times
slower)."""
import re

import pytest

from tests.test_codegen_host import _compile_asm, _kernels


def test_gated_decode_m0_only_feeds_our_lds_loads(tmp_path_factory):
    text = _compile_asm(tmp_path_factory, "gemv_gated.hip")
    for name, body in _kernels(text, "gemv_rows_kernel", 15).items():
        lines = [ln.strip() for ln in body.splitlines() if ln.strip() and not ln.strip().startswith(";")]
        assert "global_load_lds" in body, name
        for i, ln in enumerate(lines):
            if "m0" in ln:
                assert ln.startswith("s_mov_b32 m0, s"), (name, ln)
                assert lines[i + 1].startswith("global_load_lds"), (name, ln, lines[i + 1])


# norm: up to 48 blocks of 1024 without spills but for the fullest forms of 25 blocks
# and more; every adapter kernel
@pytest.mark.parametrize("src,kernels", [
    ("lora.hip", r"lora_(shrink|expand)_kernel"),
    ("norm_rotate.hip", r"norm_rotate_kernelILi[12]E"),
])
def test_no_scratch(tmp_path_factory, src, kernels):
    text = _compile_asm(tmp_path_factory, src)
    sizes = dict(re.findall(r"\.amdhsa_kernel (\S+)\n(?:.*\n)*?\s*\.amdhsa_private_segment_fixed_size (\d+)", text))
    found = {k: int(v) for k, v in sizes.items() if re.search(kernels, k)}
    assert len(found) >= 8
    assert not any(found.values()), {k: v for k, v in found.items() if v}
