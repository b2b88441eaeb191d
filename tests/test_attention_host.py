"""Host-side checks of the entry points of a block's attention half that need no GPU: bad
arguments are refused before the device is touched, with the message naming the argument,
and empty calls enqueue nothing."""
import os

import pytest

twl = pytest.importorskip("ternary_weight_linear_block_amd")
from ternary_weight_linear_block_amd import _lib  # noqa: E402

EINVAL, ESHAPE, EALIGN = 1, 2, 3
# 16-byte aligned addresses far apart, never dereferenced: every call below
# fails host validation or reaches the device query, which this host fails
P = [0x10000000 * (i + 1) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libtwl.so is not built; run `python -m ternary_weight_linear_block_amd.build`")
    return _lib.load()


def _int8(lib, **kw):
    a = dict(x_i8=P[0], a_scale=P[1], w_i8=P[2], w_scale=P[3], bias=P[4], M=4, N=100, K=1008, out=P[5], kind=_lib.OUT_BF16,
             workspace=P[6], workspace_bytes=1 << 24, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.twl_int8_linear(*a.values())


def _rope(lib, **kw):
    a = dict(qkv=P[0], kind=_lib.OUT_BF16, row_stride=1024, q_weight=P[1], k_weight=P[2], eps=1e-6, cos_sin=P[3], n_pos=100, rot=128,
             interleaved=0, positions=P[4], slots=P[5], M=4, n_q=4, n_kv=2, D=128, q=P[6], k_cache=P[7], v_cache=P[8], n_pages=10,
             page=16, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.twl_qk_norm_rope(*a.values())


def _attention(lib, **kw):
    a = dict(q=P[0], k_cache=P[1], v_cache=P[2], page_table=P[3], q_start=P[4], kv_len=P[5], scale=0.1, window=0, sinks=0, T=4, B=2,
             n_q=4, n_kv=2, D=128, n_pages=10, page=16, table_pages=8, out=P[6], workspace=P[7], workspace_bytes=1 << 24, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.twl_window_attention(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(K=0), ESHAPE, b"K="),
    (dict(K=1000), ESHAPE, b"K="),
    (dict(K=(1 << 16) + 16), ESHAPE, b"K="),
    (dict(M=-1), EINVAL, b"M="),
    (dict(N=-5), EINVAL, b"N="),
    (dict(M=(1 << 24) + 1), ESHAPE, b"M="),
    (dict(N=(1 << 24) + 1), ESHAPE, b"N="),
    (dict(M=1 << 17, N=(1 << 16) + 1), ESHAPE, b"2^33"),
    (dict(kind=_lib.OUT_ACC_I32), EINVAL, b"bias"),
    (dict(kind=7), EINVAL, b"kind"),
    (dict(x_i8=None), EINVAL, b"x_i8 is NULL"),
    (dict(w_i8=None), EINVAL, b"w_i8 is NULL"),
    (dict(out=None), EINVAL, b"out is NULL"),
    (dict(a_scale=None), EINVAL, b"a_scale is NULL"),
    (dict(w_scale=None), EINVAL, b"w_scale is NULL"),
    (dict(x_i8=P[0] + 8), EALIGN, b"x_i8"),
    (dict(w_scale=P[3] + 4), EALIGN, b"w_scale"),
    (dict(bias=P[4] + 4), EALIGN, b"bias"),
    (dict(out=P[5] + 2), EALIGN, b"out"),
    (dict(out=P[0] + 4 * 1008 - 16), EINVAL, b"out overlaps x_i8"),
    (dict(out=P[1]), EINVAL, b"out overlaps a_scale"),
    (dict(out=P[2] - 16), EINVAL, b"out overlaps w_i8"),
    (dict(out=P[3]), EINVAL, b"out overlaps w_scale"),
    (dict(out=P[4]), EINVAL, b"out overlaps bias"),
])
def test_int8_refuses(lib, kw, status, word):
    assert _int8(lib, **kw) == status
    assert word in lib.twl_last_error()


def test_int8_accepts_on_the_host(lib):
    refused = (EINVAL, ESHAPE, EALIGN)
    assert _int8(lib) not in refused
    assert _int8(lib, bias=None, kind=_lib.OUT_F32) not in refused
    assert _int8(lib, kind=_lib.OUT_ACC_I32, a_scale=None, w_scale=None, bias=None) not in refused
    assert _int8(lib, out=P[0] + 4 * 1008) not in refused  # next to each other
    assert _int8(lib, M=0, x_i8=None, a_scale=None, w_i8=None, w_scale=None, bias=None, out=None) == 0
    assert _int8(lib, N=0, out=None) == 0


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), EINVAL, b"M="),
    (dict(M=1 << 26), ESHAPE, b"M="),
    (dict(D=96), ESHAPE, b"head size"),
    (dict(n_q=5), ESHAPE, b"n_q=5"),
    (dict(n_kv=0), ESHAPE, b"n_kv=0"),
    (dict(n_q=1), ESHAPE, b"n_q=1"),
    (dict(n_q=1026, n_kv=1, row_stride=1028 * 128), ESHAPE, b"n_q=1026"),
    (dict(page=24), ESHAPE, b"page size"),
    (dict(page=0), ESHAPE, b"page size"),
    (dict(page=2048), ESHAPE, b"page size"),
    (dict(n_pages=-1), EINVAL, b"n_pages"),
    (dict(n_pages=1 << 27, page=16), ESHAPE, b"slots"),
    (dict(kind=_lib.OUT_ACC_I32), EINVAL, b"kind"),
    (dict(row_stride=1016), ESHAPE, b"row_stride"),
    (dict(row_stride=1028), ESHAPE, b"row_stride"),
    (dict(row_stride=(1 << 30) + 8), ESHAPE, b"row_stride"),
    (dict(eps=0.0), EINVAL, b"eps"),
    (dict(eps=1e-39), EINVAL, b"eps"),
    (dict(eps=float("nan")), EINVAL, b"eps"),
    (dict(eps=1e39), EINVAL, b"eps"),
    (dict(rot=8), ESHAPE, b"rot"),
    (dict(rot=144), ESHAPE, b"rot"),
    (dict(rot=-16), ESHAPE, b"rot"),
    (dict(n_pos=-1), EINVAL, b"n_pos"),
    (dict(interleaved=2), EINVAL, b"interleaved"),
    (dict(qkv=None), EINVAL, b"qkv is NULL"),
    (dict(q=None), EINVAL, b"q is NULL"),
    (dict(k_cache=None), EINVAL, b"k_cache is NULL"),
    (dict(v_cache=None), EINVAL, b"v_cache is NULL"),
    (dict(cos_sin=None), EINVAL, b"cos_sin is NULL"),
    (dict(positions=None), EINVAL, b"positions is NULL"),
    (dict(qkv=P[0] + 8), EALIGN, b"qkv"),
    (dict(slots=P[5] + 4), EALIGN, b"slots"),
    (dict(k_weight=P[2] + 2), EALIGN, b"k_weight"),
    (dict(q=P[0]), EINVAL, b"q overlaps qkv"),
    (dict(k_cache=P[6]), EINVAL, b"k_cache overlaps q"),
    (dict(v_cache=P[7] + 10 * 16 * 256 * 2 - 16), EINVAL, b"v_cache overlaps k_cache"),
    (dict(k_cache=P[3]), EINVAL, b"k_cache overlaps cos_sin"),
    (dict(v_cache=P[4]), EINVAL, b"v_cache overlaps positions"),
    (dict(q=P[5]), EINVAL, b"q overlaps slots"),
])
def test_rope_refuses(lib, kw, status, word):
    assert _rope(lib, **kw) == status
    assert word in lib.twl_last_error()


def test_rope_accepts_on_the_host(lib):
    refused = (EINVAL, ESHAPE, EALIGN)
    assert _rope(lib) not in refused
    assert _rope(lib, q_weight=None, k_weight=None, slots=None) not in refused
    assert _rope(lib, rot=0, cos_sin=None, positions=None, kind=_lib.OUT_F32, row_stride=4096) not in refused
    assert _rope(lib, v_cache=P[7] + 10 * 16 * 256 * 2) not in refused
    assert _rope(lib, n_pages=0, n_pos=0, interleaved=1) not in refused
    assert _rope(lib, M=0, qkv=None, q=None, k_cache=None, v_cache=None, cos_sin=None, positions=None) == 0


@pytest.mark.parametrize("kw,status,word", [
    (dict(T=-1), EINVAL, b"T="),
    (dict(B=-1), EINVAL, b"B="),
    (dict(T=(1 << 25) + 1), ESHAPE, b"T="),
    (dict(B=65537), ESHAPE, b"B=65537"),
    (dict(B=8192, n_q=1024, n_kv=1024), ESHAPE, b"B n_kv"),
    (dict(table_pages=-1), EINVAL, b"table_pages"),
    (dict(table_pages=(1 << 26) + 1), ESHAPE, b"table_pages"),
    (dict(n_pages=-1), EINVAL, b"n_pages"),
    (dict(n_pages=1 << 27), ESHAPE, b"slots"),
    (dict(page=8), ESHAPE, b"page size"),
    (dict(page=48), ESHAPE, b"page size"),
    (dict(D=80), ESHAPE, b"head size"),
    (dict(n_q=3), ESHAPE, b"n_q=3"),
    (dict(window=-1), EINVAL, b"window"),
    (dict(sinks=-1), EINVAL, b"sinks"),
    (dict(window=(1 << 30) + 1), ESHAPE, b"window"),
    (dict(scale=float("nan")), EINVAL, b"scale"),
    (dict(scale=float("inf")), EINVAL, b"scale"),
    (dict(scale=3e38), EINVAL, b"scale"),
    (dict(q=None), EINVAL, b"q is NULL"),
    (dict(k_cache=None), EINVAL, b"k_cache is NULL"),
    (dict(v_cache=None), EINVAL, b"v_cache is NULL"),
    (dict(page_table=None), EINVAL, b"page_table is NULL"),
    (dict(q_start=None), EINVAL, b"q_start is NULL"),
    (dict(kv_len=None), EINVAL, b"kv_len is NULL"),
    (dict(out=None), EINVAL, b"out is NULL"),
    (dict(q=P[0] + 8), EALIGN, b"q is not"),
    (dict(kv_len=P[5] + 4), EALIGN, b"kv_len"),
])
def test_attention_refuses(lib, kw, status, word):
    assert _attention(lib, **kw) == status
    assert word in lib.twl_last_error()


def test_attention_accepts_on_the_host(lib):
    refused = (EINVAL, ESHAPE, EALIGN)
    assert _attention(lib) not in refused
    assert _attention(lib, n_pages=0, k_cache=None, v_cache=None, page_table=None) not in refused
    assert _attention(lib, table_pages=0, page_table=None) not in refused
    assert _attention(lib, window=1 << 30, sinks=1 << 30, scale=-1.0, B=65536) not in refused
    assert _attention(lib, T=0, q=None, out=None) == 0
    assert _attention(lib, B=0, q_start=None, kv_len=None) == 0


def test_workspace_queries_of_invalid_sizes(lib):
    assert lib.twl_int8_workspace_bytes(4, 100, 1000) == 0
    assert lib.twl_attention_workspace_bytes(4, 2, 4, 3, 128, 16, 8, 0, 0) == 0
    assert lib.twl_attention_workspace_bytes(4, 2, 4, 2, 128, 8, 8, 0, 0) == 0
