"""qk_norm_rope where a wave takes two pieces of a token's row: both types, both pairings, numbers of
pieces that are odd (the last wave's second piece lies past the row) and last pieces that
end inside a wave.  Oracle and bound are those of test_gpu_rope.py."""
import numpy as np
import pytest

from tests import test_gpu_rope as R
from tests.gpu_helpers import announce, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def twl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_weight_linear_block_amd as m
    m.library()
    return m


def _tokens(D, n_q, n_kv):
    """Just enough of them: 64 pieces for each CU, a piece being 512 elements of a token's row."""
    pieces = -(-(n_q + 2 * n_kv) * D // 512)
    return -(-64 * torch.cuda.get_device_properties(0).multi_processor_count // pieces)


# pieces: 7, 3 (the last half full), 14, 3 (the last a quarter full), 14, 3 (half full), 1
SHAPES = [(64, 40, 8, 64), (64, 16, 2, 32), (128, 40, 8, 128), (128, 7, 1, 48), (256, 20, 4, 64), (256, 3, 1, 256), (64, 4, 2, 16)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("D,n_q,n_kv,rot", SHAPES)
def test_values(twl, D, n_q, n_kv, rot, dtype, interleaved):
    M = _tokens(D, n_q, n_kv)
    announce(f"qk_norm_rope {M} tokens {n_q}/{n_kv} x {D} rot {rot} {dtype} interleaved {interleaved}")
    c = R._case(D + rot, M, n_q, n_kv, D, rot, dtype, page=64)
    out, before = R._run(twl, c, n_q, n_kv, interleaved=interleaved)
    R._check(c, out, before, n_q, n_kv, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("D,n_q,n_kv", [(64, 40, 8), (128, 7, 1), (256, 3, 1)])
def test_padding_rows_apart_and_guards(twl, D, n_q, n_kv, dtype):
    M, width = _tokens(D, n_q, n_kv), (n_q + 2 * n_kv) * D
    c = R._case(5, M, n_q, n_kv, D, D, dtype)
    wide = torch.full((M, width + 24), float("nan"), device="cuda").to(dtype)
    wide[:, 16:16 + width] = c["qkv"]
    c["qkv"] = wide[:, 16:16 + width]
    pos, slots = host(c["positions"]).copy(), host(c["slots"]).copy()
    pos[::5], pos[1::7], slots[2::3] = -1, 500, -1
    slots[7], slots[8] = c["k_cache"].shape[0] * 16, 2 ** 31 - 1
    c["positions"], c["slots"] = dev(pos), dev(slots)
    pad = torch.full((M + 2, n_q, D), 3.0, device="cuda").bfloat16()
    q = pad[1:M + 1]
    out, before = R._run(twl, c, n_q, n_kv, q=q)
    written = (pos >= 0) & (pos < 500)
    stored = written & (slots >= 0) & (slots < c["k_cache"].shape[0] * 16)
    R._check(c, out, before, n_q, n_kv, written=written, stored=stored)
    assert (q[torch.from_numpy(~written).cuda()] == 3).all() and (pad[0] == 3).all() and (pad[-1] == 3).all()


@pytest.mark.parametrize("D,n_q,n_kv", [(64, 40, 8), (128, 7, 1), (256, 3, 1)])
def test_as_few_tokens_do(twl, D, n_q, n_kv):
    """The bits of calls that are too small for two pieces a wave, and of a side stream."""
    M = _tokens(D, n_q, n_kv)
    c = R._case(6, M, n_q, n_kv, D, D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = dict(q_weight=c["q_weight"], k_weight=None)
    many = twl.qk_norm_rope(c["qkv"], c["positions"], c["cos_sin"], n_q, n_kv, stream=side, **args)
    torch.cuda.current_stream().wait_stream(side)
    for rows in (slice(0, 100), slice(M - 101, M)):
        few = twl.qk_norm_rope(c["qkv"][rows], c["positions"][rows].clone(), c["cos_sin"], n_q, n_kv, **args)
        assert all(torch.equal(a[rows], b) for a, b in zip(many, few))
