"""The distances that written-out instructions need in the generated gfx950 code (the package's
codegen.py, which the build runs): on the library's sources, on code with a distance taken
away, and on short texts for each rule, through branches and around loops."""
import os
import re
import shutil

import pytest

from tests.test_codegen_host import _compile_asm
from ternary_weight_linear_block_amd import build as B
from ternary_weight_linear_block_amd import codegen

PRODUCT = "v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]"


def _check(*lines):
    return codegen.check("_Z1kv: ; @k\n" + "\n".join(lines) + "\n.Lfunc_end0:\n")


@pytest.fixture(scope="module")
def attention(tmp_path_factory):
    return _compile_asm(tmp_path_factory, "attention.hip")


def test_attention(attention):
    products, loads = codegen.check(attention)
    assert products >= 4 * 32 and loads >= 100


def test_int8_linear(tmp_path_factory):
    assert codegen.check(_compile_asm(tmp_path_factory, "int8_linear.hip"))[1] >= 300


def test_a_wait_taken_away_shows(attention):
    """Behind the products of a block, and before those of the last one."""
    for taken in (("s_nop 15\n\ts_nop 3", "s_nop 15\n\ts_nop 15"), ("s_nop 1\n\tv_mfma",)):
        text = attention
        for wait in taken:
            assert wait in text
            text = text.replace(wait, "v_mfma" if wait.endswith("v_mfma") else "")
        with pytest.raises(RuntimeError, match="attention_large_kernelILi256E"):
            codegen.check(text)


@pytest.mark.parametrize("use", ["v_accvgpr_read_b32 v9, a3", "v_accvgpr_write_b32 a3, v9", "global_store_dword v8, a15, s[0:1]",
                                 "v_accvgpr_mov_b32 a20, a0", "v_mfma_f32_32x32x16_bf16 a[8:23], v[0:3], v[4:7], a[8:23]"])
def test_result(use):
    with pytest.raises(RuntimeError, match=re.escape(use.split(",")[0])):
        _check(PRODUCT, "s_nop 15", "s_nop 1", use)
    if not use.startswith("v_mfma"):
        assert _check(PRODUCT, "s_nop 15", "s_nop 2", use) == (1, 0)
    assert _check(PRODUCT, PRODUCT, "v_accvgpr_read_b32 v9, a16") == (2, 0)  # the same sums again, and others


def test_operand():
    for write in ("v_mov_b32 v3, 0", "v_cvt_pk_bf16_f32 v7, v8, v9", "v_accvgpr_write_b32 a15, v9", "v_accvgpr_mov_b32 a0, a20"):
        for between in ((), ("s_waitcnt lgkmcnt(0)",)):
            with pytest.raises(RuntimeError, match="v_mfma"):
                _check(write, *between, PRODUCT)
        assert _check(write, "s_nop 1", PRODUCT) == (1, 0)
    assert _check("v_mov_b32 v8, v3", PRODUCT) == (1, 0)


def test_address():
    load = "global_load_lds_dwordx4 v1, s[4:5]"
    for write in ("v_readfirstlane_b32 s5, v2", "v_readlane_b32 s4, v2, 3"):
        with pytest.raises(RuntimeError, match="global_load_lds"):
            _check(write, "s_nop 2", "s_mov_b32 m0, s9", load)
        assert _check(write, "s_nop 3", "s_mov_b32 m0, s9", load) == (0, 1)
    assert _check("v_readfirstlane_b32 s5, v2", "s_add_u32 s5, s5, s7", "s_mov_b32 m0, s9", load) == (0, 1)


def test_around_a_loop():
    """A write at a loop's end before a product at its head, and a product at its end before a use there."""
    with pytest.raises(RuntimeError, match="v_mfma"):
        _check(".LBB0_1:", PRODUCT, "s_nop 15", "s_nop 3", "v_mov_b32 v0, 0", "s_cbranch_scc1 .LBB0_1", "s_endpgm")
    with pytest.raises(RuntimeError, match="v_accvgpr_read"):
        _check(".LBB0_1:", "v_accvgpr_read_b32 v9, a0", PRODUCT, "s_nop 15", "s_cbranch_scc1 .LBB0_1", "s_endpgm")
    assert _check(".LBB0_1:", "v_accvgpr_read_b32 v9, a0", PRODUCT, "s_nop 15", "s_nop 1", "s_cbranch_scc1 .LBB0_1", "s_endpgm") == (1, 0)


def test_through_branches():
    skip = ["s_cbranch_vccz .LBB0_2", "s_nop 15", "s_nop 15", ".LBB0_2:", "v_accvgpr_read_b32 v9, a0", "s_endpgm"]
    with pytest.raises(RuntimeError, match="v_accvgpr_read"):
        _check(PRODUCT, *skip)
    assert _check(PRODUCT, "s_nop 15", "s_nop 3", *skip) == (1, 0)
    # behind an unconditional branch nothing comes from above
    assert _check(PRODUCT, "s_branch .LBB0_2", "v_accvgpr_read_b32 v9, a0", ".LBB0_2:", "s_endpgm") == (1, 0)


def test_the_build_refuses_what_is_too_close(tmp_path, monkeypatch):
    if not os.path.exists(shutil.which("hipcc") or "/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    source = tmp_path / "csrc"
    shutil.copytree(B.CSRC, source)
    text = (source / "attention.hip").read_text()
    assert text.count("s_nop 1\\n\\tv_mfma") == 1
    (source / "attention.hip").write_text(text.replace("s_nop 1\\n\\tv_mfma", "v_mfma"))
    (tmp_path / "out").mkdir()
    monkeypatch.setattr(B, "CSRC", str(source))
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "out"))
    with pytest.raises(RuntimeError, match="attention_large_kernelILi256E"):
        B._compile("attention.hip", False)
    assert os.listdir(tmp_path / "out") == []
    (source / "attention.hip").write_text(text)
    assert os.path.exists(B._compile("attention.hip", False))


def test_sources_with_instructions_written_out_are_checked():
    for name in B.SOURCES:
        with open(os.path.join(B.CSRC, name)) as f:
            text = f.read()
        if "gemv_rows.h" in text or re.search(r'"[^"\n]*(global_load_lds|v_mfma)', text):
            assert name in B.CHECKED
