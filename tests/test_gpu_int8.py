"""int8_linear on the GPU: sums exact, outputs against the float64 oracle.

The bound.  u = 2^-24.  acc (at most 2^30) is rounded to fp32 (u), times a_scale (u), times
w_scale (u): 3 u of the product's magnitude (and 3 u^2 and less, covered by 4 u); the bias
adds one rounding of the result (u); bf16 one more of 2^-8 relative."""
import numpy as np
import pytest

import oracle.attention_oracle as A
from tests.gpu_helpers import announce, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def twl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_weight_linear_block_amd as m
    m.library()
    return m


def _case(seed, M, N, K):
    rng = np.random.default_rng(seed)
    return (rng.integers(-128, 128, (M, K), np.int8), rng.uniform(0.01, 2.0, M).astype(np.float32),
            rng.integers(-128, 128, (N, K), np.int8), rng.uniform(0.01, 2.0, N).astype(np.float32), rng.standard_normal(N).astype(np.float32) * 100)


def _compare(out, want, mag, dtype):
    tol = 4 * U * mag + U * np.abs(want)
    if dtype == torch.bfloat16:
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    got = host(out.float()).astype(np.float64)
    assert (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))


# one token to many, N and K of every remainder, the kernels' tile borders on both sides
SIZES = [(1, 1, 16), (1, 5120, 5120), (2, 17, 48), (3, 4001, 2064), (8, 64, 1024), (16, 333, 80), (17, 1000, 512), (24, 4096, 1040),
         (32, 100, 4096), (33, 257, 2064), (48, 2048, 528), (63, 70, 65536), (64, 4100, 1024), (65, 129, 4112), (100, 40, 112), (127, 640, 5120),
         (128, 255, 144), (129, 513, 2048), (200, 1028, 1008), (255, 256, 64), (256, 256, 256), (257, 260, 272), (300, 1030, 1024),
         (513, 385, 640), (700, 1999, 1072), (1024, 520, 128), (1500, 1027, 2064)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_values(twl, M, N, K):
    announce(f"int8_linear {M} x {K} -> {N}")
    x, a, w, s, bias = _case(M * 7 + N, M, N, K)
    dx, da, dw, ds, db = map(dev, (x, a, w, s, bias))
    acc, y, mag = A.int8_linear(x, a, w, s)
    assert np.array_equal(host(twl.int8_linear(dx, None, dw, None, out_dtype=torch.int32)), acc)
    for dtype in (torch.float32, torch.bfloat16):
        _compare(twl.int8_linear(dx, da, dw, ds, out_dtype=dtype), y, mag, dtype)
        _compare(twl.int8_linear(dx, da, dw, ds, bias=db, out_dtype=dtype), y + bias.astype(np.float64), mag, dtype)


@pytest.mark.parametrize("M,N", [(1, 33), (40, 100), (300, 300)])
def test_largest_sums(twl, M, N):
    K = 65536
    x, w = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
    w[1::2] = 127
    out = host(twl.int8_linear(dev(x), None, dev(w), None, out_dtype=torch.int32))
    assert (out[:, ::2] == 2 ** 30).all() and (out[:, 1::2] == -128 * 127 * K).all()


@pytest.mark.parametrize("M,N,K", [(5, 77, 1024), (90, 300, 2048), (600, 700, 1024)])
def test_scales_not_finite_stay_in_their_row_and_column(twl, M, N, K):
    x, a, w, s, bias = _case(3, M, N, K)
    a[2], s[5], bias[9] = np.nan, np.inf, np.nan
    out = host(twl.int8_linear(dev(x), dev(a), dev(w), dev(s), bias=dev(bias)))
    a2, s2, b2 = a.copy(), s.copy(), bias.copy()
    a2[2], s2[5], b2[9] = 1, 1, 1
    want = host(twl.int8_linear(dev(x), dev(a2), dev(w), dev(s2), bias=dev(b2)))
    hit = np.zeros((M, N), bool)
    hit[2], hit[:, 5], hit[:, 9] = True, True, True
    assert not np.isfinite(out[hit]).any() and np.array_equal(out[~hit], want[~hit])


@pytest.mark.parametrize("M", [4, 100, 400])
def test_rows_of_the_rotation_and_weights_made_by_it(twl, M):
    """A layer of its own: weights through rotate_quant_act; the product of the unrotated
    matrices is near (two int8 roundings: about 1e-2 of the result's norm)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, 2048, generator=g, device="cuda").bfloat16()
    w = torch.randn(500, 2048, generator=g, device="cuda").bfloat16()
    sign = (2 * torch.randint(0, 2, (2048,), generator=g, device="cuda") - 1).to(torch.int8)
    x_i8, a = twl.rotate_quant_act(x, sign)
    w_i8, s = twl.rotate_quant_act(w, sign)
    y = twl.int8_linear(x_i8, a, w_i8, s)
    _, want, mag = A.int8_linear(host(x_i8), host(a), host(w_i8), host(s))
    _compare(y, want, mag, torch.float32)
    full = host(x.double()) @ host(w.double()).T
    assert np.linalg.norm(host(y) - full) < 0.03 * np.linalg.norm(full)


@pytest.mark.parametrize("M,N,K", [(1, 100, 512), (40, 1000, 4096), (300, 500, 5120)])
def test_guard_rows_stream_and_garbage_workspace(twl, M, N, K):
    x, a, w, s, _ = _case(11, M, N, K)
    dx, da, dw, ds = map(dev, (x, a, w, s))
    need = twl.int8_workspace_bytes(M, N, K)
    pad = torch.full((M * N + 1024,), 7.0, device="cuda")
    out = pad[512:512 + M * N].view(M, N)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert twl.int8_linear(dx, da, dw, ds, out=out, workspace=ws, stream=side) is out
    torch.cuda.current_stream().wait_stream(side)
    _, want, mag = A.int8_linear(x, a, w, s)
    _compare(out, want, mag, torch.float32)
    assert (pad[:512] == 7).all() and (pad[512 + M * N:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(1, 5120, 5120), (24, 1024, 4096), (100, 512, 5120), (400, 700, 2048)])
def test_graph_replays(twl, M, N, K):
    x, a, w, s, _ = _case(13, M, N, K)
    dx, da, dw, ds = map(dev, (x, a, w, s))
    twl.int8_linear(dx, da, dw, ds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = twl.int8_linear(dx, da, dw, ds)
    for r in range(3):
        dx.copy_(torch.roll(dx, r + 1, 0))
        eager = twl.int8_linear(dx, da, dw, ds)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_empty(twl):
    x, a = torch.zeros((0, 64), dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda")
    w, s = torch.zeros((5, 64), dtype=torch.int8, device="cuda"), torch.zeros(5, device="cuda")
    assert twl.int8_linear(x, a, w, s).shape == (0, 5)
    assert twl.int8_linear(w, s, x, a).shape == (5, 0)


def test_refusals(twl):
    x, a, w, s, bias = map(dev, _case(1, 4, 6, 64))
    with pytest.raises(ValueError, match="a_scale"):
        twl.int8_linear(x, a[:3], w, s)
    with pytest.raises(ValueError, match="w_i8"):
        twl.int8_linear(x, a, w[:, :32], s)
    with pytest.raises(TypeError, match="out_dtype"):
        twl.int8_linear(x, a, w, s, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="requires grad"):
        twl.int8_linear(x, a.clone().requires_grad_(), w, s)
    with pytest.raises(twl.TwlError, match="bias"):
        twl.int8_linear(x, a, w, s, bias=bias, out_dtype=torch.int32)
    with pytest.raises(twl.TwlError, match="K="):
        twl.int8_linear(x[:, :40].contiguous(), a, w[:, :40].contiguous(), s)
    with pytest.raises(ValueError, match="on the GPU"):
        twl.int8_linear(x, a, w.cpu(), s)
