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


def _registers(text):
    """The accumulation ('a') and vector ('v') registers that an operand text names."""
    out = set()
    for kind, first, last in re.findall(r"\b([av])\[(\d+):(\d+)\]", text):
        out |= {(kind, r) for r in range(int(first), int(last) + 1)}
    return out | {(kind, int(r)) for kind, r in re.findall(r"\b([av])(\d+)\b", text)}


def test_accumulation_registers_of_the_wide_heads(tmp_path_factory):
    """The kernel of 256-wide heads has its matrix products on accumulation registers written out, which the
    compiler knows nothing of: nothing else may touch such a register, nor a path leave the block of code, within 19
    states behind the product that writes it (16 passes and 3), and no product may read what an operation wrote less
    than 2 states before."""
    kernels = _kernels(_compile_asm(tmp_path_factory, "attention.hip"), "attention_large_kernel", 3)
    body = next(b for k, b in kernels.items() if "ILi256E" in k)
    now, product, written, products = 0, {}, {}, 0
    for raw in body.splitlines():
        ln = raw.strip()
        if re.match(r"\.LBB|; %bb", raw) or ln.startswith(("s_cbranch", "s_branch", "s_endpgm")):
            assert not [r for r, t in product.items() if now - t < 19], ln
            product = {}
            now += 1
            continue
        if not ln or ln.startswith((";", ".")):
            continue
        dest, _, rest = ln.partition(",")
        if re.match(r"v_mfma\S+ a\[", ln):
            assert not [r for r in _registers(rest) if now - written.get(r, -99) < 2], ln
            product.update({r: now for r in _registers(dest)})
            products += 1
        elif ln.startswith("s_nop"):
            now += int(ln.split()[1])
        else:
            assert not [r for r in _registers(ln) if now - product.get(r, -99) < 19], ln
            if ln.startswith("v_"):
                written.update({r: now for r in _registers(dest)})
        now += 1
    assert products >= 4 * 32
