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


def _scratch(text):
    return {k: int(v) for k, v in
            re.findall(r"\.amdhsa_kernel (\S+)\n(?:.*\n)*?\s*\.amdhsa_private_segment_fixed_size (\d+)", text)}


def test_lora_token_kernel_has_no_scratch(tmp_path_factory):
    sizes = {k: v for k, v in _scratch(_compile_asm(tmp_path_factory, "lora.hip")).items() if "lora_token_kernel" in k}
    assert len(sizes) == 2 and not any(sizes.values()), sizes


def test_norm_forms_that_are_launched(tmp_path_factory):
    """The split for many tokens of the norm alone (two blocks a wave, 256 threads) is
    built without a branch only."""
    names = _scratch(_compile_asm(tmp_path_factory, "norm_rotate.hip"))
    forms = [re.search(r"norm_rotate_kernelILi(\d)ELb(\d)ELb(\d)ELb(\d)ELi(\d+)E", k).groups() for k in names]
    assert len(forms) == 18
    assert sorted(f for f in forms if f[4] == "256") == [("2", "0", "0", "0", "256"), ("2", "1", "0", "0", "256")]
