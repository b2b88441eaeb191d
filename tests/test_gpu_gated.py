"""pack_ternary_gated and ternary_gated_linear on the GPU against the oracle.

The bound, element by element, with u = 2^-24.  The accumulators are exact; the
rescale to g and u is three fp32 products and a conversion each (4 u); an error of
4 u in g moves SiLU(g) by at most (1 + |g|) 4 u relative; the exponential's argument
is off by |g| u, and the native exponential, the reciprocal, the sum and the
products by 8 u together: (5 |g| + 16) u relative, and the output's own rounding,
2^-8 for bf16 and u for fp32.  Where 1 + e^-g passes 2^126 its reciprocal is below
the smallest normal number 2^-126 and the native instruction returns 0, so the
product may be off by 2^-126 |g u|, and an output below 2^-126 may be flushed."""
import numpy as np
import pytest

import oracle.block_oracle as B
import oracle.twl_oracle as O
import workloads as W
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


def _case(seed, M, N, K, gain=1.0):
    gate, up = W.make_layer(seed, M, K, N), W.make_layer(seed + 1000, M, K, N, codes="sparse40")
    x_i8, a_scale = O.rotate_quant_act(gate.x_bits, gate.sign)
    return dict(x_i8=x_i8, a_scale=(a_scale * np.float32(gain)).astype(np.float32), gate=gate, up=up)


def _pack(twl, c):
    g, u = c["gate"], c["up"]
    return twl.pack_ternary_gated(dev(g.code), dev(g.s_bits.view(np.int16)), dev(u.code), dev(u.s_bits.view(np.int16)))


def _want(c):
    _, qg, sg = O.pack_ternary(c["gate"].code, c["gate"].s_bits)
    _, qu, su = O.pack_ternary(c["up"].code, c["up"].s_bits)
    return B.gated_linear(c["x_i8"], c["a_scale"], c["gate"].code, qg, sg, c["up"].code, qu, su)


def _check(out, want, mag, mag_u):
    got = host(out.float()).astype(np.float64)
    tol = np.abs(want) * ((5 * mag + 16) * U + (2.0 ** -8 if out.dtype == torch.bfloat16 else U)) + 2.0 ** -126 * (1 + mag * mag_u)
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, f"{len(bad)} off, first {bad[:4].tolist()}: {got[tuple(bad[0])]!r} for {want[tuple(bad[0])]!r}"


@pytest.mark.parametrize("N,K", [(1, 1024), (33, 2048), (130, 1024)])
def test_pack(twl, N, K):
    c = _case(N, 1, N, K)
    code = np.stack([c["gate"].code, c["up"].code], 1).reshape(2 * N, K)
    s = np.stack([c["gate"].s_bits, c["up"].s_bits], 1).reshape(2 * N, K // 128)
    announce(f"pack gated N={N} K={K}")
    packed, q, smax = _pack(twl, c)
    op, oq, osm = O.pack_ternary(code, s)
    assert np.array_equal(host(packed).reshape(-1), np.asarray(op).reshape(-1))
    assert np.array_equal(host(q), oq)
    assert np.array_equal(host(smax).view(np.uint32), osm.view(np.uint32))
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    c["gate"].code[0, 3] = 5
    c["up"].code[N - 1, 9] = -7
    g, u = c["gate"], c["up"]
    twl.pack_ternary_gated(dev(g.code), dev(g.s_bits.view(np.int16)), dev(u.code), dev(u.s_bits.view(np.int16)), bad_codes=bad)
    assert bad.item() == 2


# narrow layers (finishing kernel; odd widths), the row-balanced kernel from 2048
# columns on, every token form of it, GEMM tiles and splits, odd and ragged
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1024), (2, 65, 2048), (3, 333, 1024), (5, 1001, 2048), (24, 500, 5120), (17, 2047, 1024),
    (1, 2048, 1024), (4, 2051, 1024), (16, 4001, 2048), (24, 4350, 1024), (20, 8704, 1024), (8, 12299, 1024),
    (1, 2200, 17408), (24, 2050, 17408), (9, 2048, 33792),
    (25, 1, 1024), (25, 77, 2048), (130, 1002, 1024), (77, 4001, 2048), (300, 2560, 2048), (64, 640, 17408)])
def test_values(twl, M, N, K):
    c = _case(M + N, M, N, K)
    packed, q, smax = _pack(twl, c)
    x, a = dev(c["x_i8"]), dev(c["a_scale"])
    want, mag, mag_u = _want(c)
    announce(f"gated M={M} N={N} K={K}")
    out = twl.ternary_gated_linear(x, a, packed, q, smax, out_dtype=torch.float32)
    _check(out, want, mag, mag_u)
    assert torch.equal(twl.ternary_gated_linear(x, a, packed, q, smax), out.bfloat16())
    for path in (twl.PATH_GEMM,) + ((twl.PATH_GEMV,) if M <= twl.GEMV_MAX_M else ()):
        announce(f"gated M={M} N={N} K={K} path={path}")
        assert torch.equal(twl.ternary_gated_linear(x, a, packed, q, smax, out_dtype=torch.float32, path=path), out)


@pytest.mark.parametrize("M", [3, 40])
def test_large_gates_and_zero_rows(twl, M):
    """Gates of hundreds (e^-g overflows and underflows), a token of zeros."""
    c = _case(M, M, 2100, 1024, gain=300.0)
    c["x_i8"][1] = 0
    c["a_scale"][1] = 0.0
    packed, q, smax = _pack(twl, c)
    want, mag, mag_u = _want(c)
    assert mag.max() > 120
    announce(f"gated large M={M}")
    out = twl.ternary_gated_linear(dev(c["x_i8"]), dev(c["a_scale"]), packed, q, smax, out_dtype=torch.float32)
    assert torch.isfinite(out).all() and not out[1].any()
    _check(out, want, mag, mag_u)


def test_guards_streams_and_graphs(twl):
    """Rows behind the last and the workspace's end are left; two calls on two
    streams, two captured graphs replayed at once with changed inputs."""
    shapes = [(20, 500, 2048), (64, 640, 17408)]  # both with a workspace: slices, split-K
    cases = [_case(k, *s) for k, s in enumerate(shapes)]
    ws = [_pack(twl, c) for c in cases]
    wants = [_want(c) for c in cases]
    ins = [(dev(c["x_i8"]), dev(c["a_scale"])) for c in cases]
    for (M, N, K), (x, a), w, want in zip(shapes, ins, ws, wants):
        need = twl.gated_workspace_bytes(M, N, K)
        assert need > 0
        buf = torch.full((M + 2, N), 7.0, device="cuda")
        work = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
        announce(f"gated guards M={M} N={N}")
        _check(twl.ternary_gated_linear(x, a, *w, out=buf[:M], workspace=work), *want)
        assert torch.all(buf[M:] == 7.0).item() and torch.all(work[need:] == 0x7F).item()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    announce("gated two streams")
    outs = [twl.ternary_gated_linear(x, a, *w, stream=s) for (x, a), w, s in zip(ins, ws, streams)]
    torch.cuda.synchronize()
    for o, want in zip(outs, wants):
        _check(o, *want)
    graphs = []
    for (x, a), w in zip(ins, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = twl.ternary_gated_linear(x, a, *w)
        graphs.append((g, o))
    announce("gated two graphs")
    for k in range(3):
        for c, (x, a) in zip(cases, ins):
            c["x_i8"] = np.roll(c["x_i8"], 1, axis=0)
            c["a_scale"] = (c["a_scale"] * np.float32(1.25)).astype(np.float32)
            x.copy_(dev(c["x_i8"]))
            a.copy_(dev(c["a_scale"]))
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, o), c in zip(graphs, cases):
            _check(o, *_want(c))


def test_python_refusals(twl):
    c = _case(1, 4, 64, 1024)
    w = _pack(twl, c)
    x, a = dev(c["x_i8"]), dev(c["a_scale"])
    f = twl.ternary_gated_linear
    for args, kw in (((x.float(), a) + w, {}), ((x, a[:3]) + w, {}), ((x, a, w[0][:-64], w[1], w[2]), {}),
                     ((x, a, w[0], w[1][:-1], w[2]), {}), ((x, a, w[0], w[1], w[2][:-2]), {}),
                     ((x, a) + w, dict(out_dtype=torch.float16)), ((x, a) + w, dict(out=torch.empty((4, 63), device="cuda"))),
                     ((x, a) + w, dict(path=twl.PATH_GEMV_DOT4)), ((x.cpu(), a) + w, {}), ((x[0], a) + w, {})):
        with pytest.raises((ValueError, TypeError, twl.TwlError)):
            f(*args, **kw)
    s = dev(c["gate"].s_bits.view(np.int16))
    with pytest.raises(ValueError):
        twl.pack_ternary_gated(dev(c["gate"].code), s, dev(c["up"].code[:63]), s)
    assert f(x[:0], a[:0], *w).shape == (0, 64)


# rows of more than 33 groups a wave (K above 33792) leave the row-balanced kernel at
# any width: partial sums of slices of K and the finishing kernel
@pytest.mark.parametrize("M,N,K", [(1, 2048, 34816), (4, 2051, 34816), (24, 2048, 34816), (1, 2049, 65536), (24, 2048, 65536)])
def test_long_rows_of_wide_layers(twl, M, N, K):
    c = _case(M + K, M, N, K)
    w = _pack(twl, c)
    x, a = dev(c["x_i8"]), dev(c["a_scale"])
    assert twl.gated_workspace_bytes(M, N, K) >= 2 * M * 2 * N * 4  # two slices at least
    announce(f"gated M={M} N={N} K={K}")
    out = twl.ternary_gated_linear(x, a, *w, out_dtype=torch.float32)
    _check(out, *_want(c))
    announce(f"gated M={M} N={N} K={K} GEMM")
    assert torch.equal(twl.ternary_gated_linear(x, a, *w, out_dtype=torch.float32, path=twl.PATH_GEMM), out)
    assert torch.equal(twl.ternary_gated_linear(x, a, *w), out.bfloat16())


@pytest.mark.parametrize("M,N", [(24, 4), (24, 2048), (4096, 4)])
def test_silu_bound(twl, M, N):
    """The bound that twl.h states for the activation, (1.25 |g| + 8) 2^-24, with g
    and u exact: sums of +-1 and a smax of 127 / 128, whose 127th part is 2^-7, so g
    and u are a_scale with another exponent.  Dense around -44.38, where the
    rounding of g log2(e) and the error of its constant add up."""
    assert np.float32(127 / 128) * (np.float32(1) / np.float32(127)) == np.float32(2.0 ** -7)
    K = 1024
    gate = np.zeros((N, K), np.int8)
    up = np.zeros((N, K), np.int8)
    gate[0::2, 128], gate[1::2, 128], up[:, 128] = -1, 1, 1
    s = np.full((N, K // 128), 1 / 128, np.float16)   # q = 1 there
    s[:, 0] = 127 / 128                              # and 127 in the first group
    x = np.zeros((M, K), np.int8)
    x[:, 128] = 1
    rng = np.random.default_rng(M)
    g = np.where(rng.random(M) < 0.5, rng.uniform(44.2, 44.6, M), np.exp(rng.uniform(np.log(0.01), np.log(86), M))).astype(np.float32)
    g[0] = 44.3821
    w = twl.pack_ternary_gated(dev(gate), dev(s.view(np.int16)), dev(up), dev(s.view(np.int16)))
    announce(f"silu bound M={M} N={N}")
    out = host(twl.ternary_gated_linear(dev(x), dev(g * np.float32(128)), *w, out_dtype=torch.float32)).astype(np.float64)
    u = g.astype(np.float64)
    for row, sign in ((0, -1.0), (1, 1.0)):
        want = sign * u / (1.0 + np.exp(-sign * u)) * u
        err = np.abs(out[:, row] - want) / np.abs(want)
        over = err - (1.25 * u + 8) * U
        at = int(np.argmax(over))
        assert over[at] <= 0, (sign * u[at], err[at] / U)
        assert np.array_equal(out[:, row], out[:, row + 2])
