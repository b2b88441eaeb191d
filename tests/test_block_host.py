"""Host-side checks of the block operators' entry points that need no GPU: bad
arguments are refused before the device is touched, with the message naming
the argument, and empty calls enqueue nothing."""
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


def _norm(lib, **kw):
    a = dict(x=P[0], residual=P[1], post_weight=P[2], gate=P[3], gate_stride=0, branch_scale=1.0, weight=P[4], eps=1e-6,
             sign=P[5], M=4, K=1024, h=P[6], normed=P[7], x_i8=P[8], a_scale=P[9], stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.twl_norm_rotate_quant_act(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(K=1000), ESHAPE, b"K="),
    (dict(K=65536 + 1024), ESHAPE, b"K="),
    (dict(M=-1), EINVAL, b"M="),
    (dict(x=None), EINVAL, b"x is NULL"),
    (dict(weight=None), EINVAL, b"weight is NULL"),
    (dict(x_i8=None), EINVAL, b"x_i8 is NULL"),
    (dict(a_scale=None), EINVAL, b"a_scale is NULL"),
    (dict(x=P[0] + 8), EALIGN, b"x is not"),
    (dict(residual=P[1] + 2), EALIGN, b"residual"),
    (dict(gate=P[3] + 4), EALIGN, b"gate"),
    (dict(h=P[6] + 2), EALIGN, b"h is not"),
    (dict(eps=0.0), EINVAL, b"eps"),
    (dict(eps=float("nan")), EINVAL, b"eps"),
    (dict(eps=float("inf")), EINVAL, b"eps"),
    (dict(branch_scale=float("inf")), EINVAL, b"branch_scale"),
    (dict(gate_stride=1023), ESHAPE, b"gate_stride"),
    (dict(gate_stride=1028), ESHAPE, b"gate_stride"),
    (dict(gate_stride=-1024), ESHAPE, b"gate_stride"),
    (dict(sign=None), EINVAL, b"need sign"),
    (dict(sign=None, x_i8=None, a_scale=None, normed=None), EINVAL, b"no output"),
    (dict(residual=None, post_weight=None, gate=None), EINVAL, b"it would be x"),
    # overlaps: h may be x or residual themselves, not shifted; nothing else may
    (dict(h=P[0] + 16), EINVAL, b"h overlaps x"),
    (dict(h=P[3]), EINVAL, b"h overlaps gate"),
    (dict(normed=P[0]), EINVAL, b"normed overlaps x"),
    (dict(normed=P[6]), EINVAL, b"normed overlaps h"),
    (dict(x_i8=P[1]), EINVAL, b"x_i8 overlaps residual"),
    (dict(a_scale=P[8] + 4096 - 16), EINVAL, b"a_scale overlaps x_i8"),
])
def test_norm_refuses(lib, kw, status, word):
    assert _norm(lib, **kw) == status
    assert word in lib.twl_last_error()


def test_norm_accepts_on_the_host(lib):
    refused = (EINVAL, ESHAPE, EALIGN)
    assert _norm(lib) not in refused
    assert _norm(lib, h=P[0]) not in refused
    assert _norm(lib, h=P[1]) not in refused
    assert _norm(lib, h=None, normed=None) not in refused
    assert _norm(lib, gate_stride=2048) not in refused
    assert _norm(lib, residual=None, post_weight=None, gate=None, h=None) not in refused
    assert _norm(lib, sign=None, x_i8=None, a_scale=None) not in refused
    # the last byte of x_i8 and the first of a_scale next to each other
    assert _norm(lib, a_scale=P[8] + 4096) not in refused
    assert _norm(lib, M=0, x=None, weight=None, sign=None, h=None, normed=None, x_i8=None, a_scale=None) == 0


def _lora(lib, **kw):
    a = dict(y=P[0], x=P[1], ids=P[2], lora_a=P[3], lora_b=P[4], scale=P[5], M=4, N=64, K=1024, R=16, n_adapters=3, kind=0,
             out=P[6], workspace=P[7], workspace_bytes=1 << 20, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.twl_lora_add(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(K=1000), ESHAPE, b"K="),
    (dict(K=0), ESHAPE, b"K="),
    (dict(K=65536 + 128), ESHAPE, b"K="),
    (dict(R=4), ESHAPE, b"R="),
    (dict(R=12), ESHAPE, b"R="),
    (dict(R=136), ESHAPE, b"R="),
    (dict(R=0), ESHAPE, b"R="),
    (dict(M=-1), EINVAL, b"M="),
    (dict(N=-1), EINVAL, b"N="),
    (dict(n_adapters=-1), EINVAL, b"n_adapters="),
    (dict(kind=1), EINVAL, b"kind"),
    (dict(kind=3), EINVAL, b"kind"),
    (dict(y=None), EINVAL, b"y is NULL"),
    (dict(x=None), EINVAL, b"x is NULL"),
    (dict(ids=None), EINVAL, b"ids is NULL"),
    (dict(lora_a=None), EINVAL, b"lora_a is NULL"),
    (dict(lora_b=None), EINVAL, b"lora_b is NULL"),
    (dict(scale=None), EINVAL, b"scale is NULL"),
    (dict(out=None), EINVAL, b"out is NULL"),
    (dict(x=P[1] + 2), EALIGN, b"x is not"),
    (dict(out=P[6] + 4), EALIGN, b"out is not"),
])
def test_lora_refuses(lib, kw, status, word):
    assert _lora(lib, **kw) == status
    assert word in lib.twl_last_error()


def test_lora_empty_calls(lib):
    none = dict(y=None, x=None, ids=None, lora_a=None, lora_b=None, scale=None, out=None, workspace=None, workspace_bytes=0)
    assert _lora(lib, M=0, **none) == 0
    assert _lora(lib, N=0, **none) == 0
    # without adapters the copy needs y, ids and out only
    assert _lora(lib, n_adapters=0, x=None, lora_a=None, lora_b=None, scale=None) not in (EINVAL, ESHAPE, EALIGN)
    assert lib.twl_lora_workspace_bytes(4, 1000, 16, 1) == 0


def _gated(lib, **kw):
    a = dict(x_i8=P[0], a_scale=P[1], packed=P[2], q=P[3], smax=P[4], M=4, N=64, K=1024, out=P[5], out_kind=2, path=0,
             workspace=P[6], workspace_bytes=1 << 20, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.twl_ternary_gated_linear(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(K=1000), ESHAPE, b"K="),
    (dict(M=-1), EINVAL, b"M="),
    (dict(N=-1), EINVAL, b"N="),
    (dict(N=(1 << 29) + 1), ESHAPE, b"N="),
    (dict(out_kind=1), EINVAL, b"output kind"),
    (dict(out_kind=3), EINVAL, b"output kind"),
    (dict(path=3), EINVAL, b"path"),
    (dict(path=-1), EINVAL, b"path"),
    (dict(path=2, M=25), ESHAPE, b"M <="),
    (dict(x_i8=None), EINVAL, b"x_i8 is NULL"),
    (dict(a_scale=None), EINVAL, b"a_scale is NULL"),
    (dict(packed=None), EINVAL, b"packed is NULL"),
    (dict(q=None), EINVAL, b"q is NULL"),
    (dict(smax=None), EINVAL, b"smax is NULL"),
    (dict(out=None), EINVAL, b"out is NULL"),
    (dict(out=P[5] + 8), EALIGN, b"out is not"),
    (dict(out=P[0] + 4080), EINVAL, b"out overlaps x_i8"),
    (dict(out=P[2] - 512 + 16), EINVAL, b"out overlaps packed"),
    (dict(out=P[3] + 1008), EINVAL, b"out overlaps q"),
    (dict(out=P[4]), EINVAL, b"out overlaps smax"),
])
def test_gated_refuses(lib, kw, status, word):
    assert _gated(lib, **kw) == status
    assert word in lib.twl_last_error()


def test_gated_empty_calls_and_pack(lib):
    none = dict(x_i8=None, a_scale=None, packed=None, q=None, smax=None, out=None, workspace=None, workspace_bytes=0)
    assert _gated(lib, M=0, **none) == 0
    assert _gated(lib, N=0, **none) == 0
    pack = lib.twl_pack_ternary_gated
    assert pack(None, None, None, None, 0, 1024, None, None, None, None, None) == 0
    assert pack(P[0], P[1], P[2], P[3], 8, 1000, P[4], P[5], P[6], None, None) == ESHAPE
    assert pack(P[0], P[1], None, P[3], 8, 1024, P[4], P[5], P[6], None, None) == EINVAL
    assert b"code_up is NULL" in lib.twl_last_error()
    assert pack(P[0], P[1], P[2], P[3] + 2, 8, 1024, P[4], P[5], P[6], None, None) == EALIGN
    assert pack(P[0], P[1], P[2], P[3], 8, 1024, P[4], P[5], P[6], P[7] + 2, None) == EALIGN
    assert lib.twl_gated_workspace_bytes(4, 64, 1000) == 0


def test_tensors_that_require_grad_are_refused():
    """The operators have no backward pass: a result without a graph would lose an
    adapter's gradients without a word.  With gradients off the call goes through."""
    torch = pytest.importorskip("torch")
    from ternary_weight_linear_block_amd import block

    class OnGpu:  # what _check asks of a tensor
        def __init__(self, t):
            self.t, self.is_cuda, self.device = t, True, "cuda:0"

        def get_device(self):
            return 0

        def __getattr__(self, name):
            return getattr(self.t, name)

    w = torch.nn.Parameter(torch.zeros((3, 8), dtype=torch.bfloat16))
    args = ("lora_a", (3, 8), (torch.bfloat16,), 0)
    with pytest.raises(ValueError, match="lora_a requires grad"):
        block._check(OnGpu(w), *args)
    with pytest.raises(ValueError, match="has shape"):
        block._check(OnGpu(w), "lora_a", (3, 9), (torch.bfloat16,), 0)
    with pytest.raises(ValueError, match="contiguous"):
        block._check(OnGpu(w.t()), "lora_a", (8, 3), (torch.bfloat16,), 0)
    with torch.no_grad():
        assert block._check(OnGpu(w), *args) == w.data_ptr()
    assert block._check(OnGpu(w.detach()), *args) == w.data_ptr()
