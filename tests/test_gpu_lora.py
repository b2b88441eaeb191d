"""lora_add on the GPU against the float64 oracle, element by element.

The bound.  u = 2^-24 is fp32's unit roundoff.  A sum of n fp32 terms in any order
is off by at most n u times the sum of the magnitudes: v by K u (|x| |A|), with
the slices' sums and the scale included in K + 64.  Two (three) bf16 terms hold v to
2^-16 (2^-24) of it, and the second product sums R of each: together
2^-16 (2^-24) + (3 R + 8) u of |v| |B|.  Adding y rounds once in fp32 (u) and once
to y's type: 2^-8 for bf16, u for fp32, relative to the result."""
import numpy as np
import pytest

import oracle.block_oracle as B
from tests.gpu_helpers import announce, host

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


def _case(seed, M, N, K, R, n, dtype, ids):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    ids = np.asarray(ids(rng, M, n) if callable(ids) else ids, np.int32)
    return dict(y=t(M, N).to(dtype).cuda(), x=t(M, K).to(torch.bfloat16).cuda(), ids=torch.from_numpy(ids).cuda(),
                lora_a=(t(n, R, K) / K ** 0.5).to(torch.bfloat16).cuda(), lora_b=t(n, N, R).to(torch.bfloat16).cuda(),
                scale=torch.from_numpy(rng.uniform(0.5, 2.0, n).astype(np.float32)).cuda())


def _np(t):
    return host(t.float()).astype(np.float64)


def _check(out, c, rows=None, y=None):
    want, mag_x, mag_v = B.lora_add(_np(c["y"] if y is None else y), _np(c["x"]), host(c["ids"]), _np(c["lora_a"]),
                                    _np(c["lora_b"]), host(c["scale"]))
    K, R = c["x"].shape[1], c["lora_a"].shape[1]
    bf16 = c["y"].dtype == torch.bfloat16
    delta = (K + 64) * U * mag_x + ((2.0 ** -16 if bf16 else 2.0 ** -24) + (3 * R + 8) * U) * mag_v
    tol = delta + (np.abs(want) + delta) * ((2.0 ** -8 if bf16 else U) + U)
    got = _np(out)
    rows = range(len(got)) if rows is None else rows
    err = np.abs(got - want)[rows]
    bad = np.argwhere(~(err <= tol[rows]))
    assert bad.size == 0, f"{len(bad)} off, first {bad[:4].tolist()}, err {err[tuple(bad[0])]:.3g} tol {tol[rows][tuple(bad[0])]:.3g}"
    none = [t for t, i in enumerate(host(c["ids"])) if not 0 <= i < c["lora_a"].shape[0]]
    assert torch.equal(out[none], (c["y"] if y is None else y)[none])


def mixed(rng, M, n):
    return rng.integers(-1, n, M)


def runs(rng, M, n):
    return np.repeat(rng.integers(-1, n, M), rng.integers(1, 40, M))[:M]


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K,R,n,ids", [
    (1, 64, 1024, 8, 1, [0]),
    (1, 5120, 5120, 16, 4, [3]),
    (1, 130, 128, 16, 2, [1]),
    (3, 1, 256, 16, 2, [1, 0, 1]),
    (16, 33, 1024, 24, 3, mixed),
    (17, 1001, 2048, 40, 5, mixed),
    (24, 2048, 1024, 16, 32, mixed),
    (64, 520, 1024, 64, 3, runs),
    (65, 264, 1024, 72, 4, runs),
    (200, 1032, 2048, 128, 6, runs),
    (333, 16400, 1024, 32, 4, runs),
    (300, 16501, 256, 96, 9, mixed),
    (130, 32768, 128, 128, 2, runs),
    (128, 33000, 128, 64, 3, mixed),
    (256, 72, 512, 40, 20, mixed),
    (257, 72, 512, 40, 20, mixed),
    (700, 1032, 512, 128, 20, mixed),
    (1030, 264, 512, 64, 5, runs),
    (1040, 77, 256, 8, 3, runs),
    (1100, 136, 256, 32, 40, mixed),
    (1025, 16392, 128, 24, 6, runs),
    # rows that are no whole pieces of 16 bytes: 4-byte aligned, odd, shorter than one range
    (300, 1002, 512, 64, 5, runs),
    (400, 10713, 128, 32, 3, runs),
    (270, 66, 512, 128, 4, mixed),
    (1100, 63, 256, 16, 6, runs),
    (4200, 4099, 128, 16, 3, runs),
    (90, 4666, 2048, 32, 9, mixed),
])
def test_values(twl, M, N, K, R, n, ids, dtype):
    announce(f"lora M={M} N={N} K={K} R={R} n={n} {dtype}")
    c = _case(M + N + R, M, N, K, R, n, dtype, ids)
    _check(twl.lora_add(**c), c)


@pytest.mark.parametrize("M,N", [(5, 136), (70, 136), (260, 16384), (300, 1003), (290, 70), (333, 16386), (270, 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_and_no_adapter(twl, M, N, dtype):
    """y updated in place; every token without an adapter, also by ids out of range."""
    c = _case(M, M, N, 512, 16, 3, dtype, mixed)
    y = c["y"].clone()
    announce(f"lora in place M={M} N={N} {dtype}")
    out = twl.lora_add(out=c["y"], **c)
    assert out is c["y"]
    _check(out, c, y=y)
    c = _case(M, M, N, 512, 16, 3, dtype, [(-1, 3, 2 ** 31 - 1, -2 ** 31)[t % 4] for t in range(M)])
    announce(f"lora no adapter M={M}")
    assert torch.equal(twl.lora_add(**c), c["y"])
    empty = dict(c, lora_a=c["lora_a"][:0], lora_b=c["lora_b"][:0], scale=c["scale"][:0])
    assert torch.equal(twl.lora_add(**empty), c["y"])


def test_same_adapter_everywhere_and_twice(twl):
    """One adapter for all tokens; the same token rows twice give the same rows."""
    c = _case(1, 96, 16400, 1024, 64, 2, BF, [1] * 96)
    for k in ("x", "y"):
        c[k][48:] = c[k][:48]
    announce("lora one adapter")
    out = twl.lora_add(**c)
    _check(out, c)
    assert torch.equal(out[48:], out[:48])
    assert torch.equal(out, twl.lora_add(**c))


@pytest.mark.parametrize("M,N", [(20, 72), (80, 16392)])
def test_nan_stays_with_its_users(twl, M, N):
    """NaN and infinities in one adapter, one token and the unused adapter reach
    their own tokens' rows only."""
    ids = [t % 4 for t in range(M)]
    c = _case(M, M, N, 256, 16, 5, F32, ids)
    c["lora_a"][2, 3, 7] = float("nan")
    c["lora_b"][2, :, 1] = float("inf")
    c["lora_a"][4] = float("nan")
    c["lora_b"][4] = float("nan")
    c["x"][5] = float("inf")
    announce(f"lora nan M={M}")
    out = twl.lora_add(**c)
    fine = [t for t in range(M) if ids[t] != 2 and t != 5]
    with np.errstate(invalid="ignore"):
        _check(out, c, rows=fine)
    assert not torch.isfinite(out[2]).any()


def test_rows_behind_the_last_stay(twl):
    c = _case(4, 21, 200, 256, 16, 3, BF, mixed)
    buf = torch.full((24, 200), 7.0, dtype=BF, device="cuda")
    ws = torch.full((twl.lora_workspace_bytes(21, 256, 16, 3) + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    announce("lora guard rows")
    _check(twl.lora_add(out=buf[:21], workspace=ws, **c), c)
    assert torch.all(buf[21:] == 7.0).item()
    assert torch.all(ws[-64:] == 0x7F).item()


def test_two_streams_and_graphs(twl):
    """Calls on two streams at once, and two graphs replayed at once, keep their
    own workspaces; replays follow changed inputs and ids."""
    cases = [_case(7 + k, 200, 1024, 2048, 32, 4, F32, runs) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    announce("lora two streams")
    outs = [twl.lora_add(stream=s, **c) for s, c in zip(streams, cases)]
    torch.cuda.synchronize()
    for o, c in zip(outs, cases):
        _check(o, c)
    announce("lora two graphs")
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = twl.lora_add(**c)
        graphs.append((g, o))
    for k in range(3):
        for i, c in enumerate(cases):
            new = _case(50 + 2 * k + i, 200, 1024, 2048, 32, 4, F32, mixed if k else runs)
            for name in c:
                c[name].copy_(new[name])
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, o), c in zip(graphs, cases):
            _check(o, c)


@pytest.mark.parametrize("M,R", [(9, 16), (9, 64), (300, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tokens_without_adapter_keep_their_bits(twl, M, R, dtype):
    """NaN with any payload, infinities, denormals and minus zero are copied."""
    N = 90
    c = _case(M, M, N, 256, R, 3, dtype, [(-1, 1, 7)[t % 3] for t in range(M)])
    if dtype == BF:
        bits = torch.tensor([0x7F81, -0x0001, 0x7F80, -0x0080, 0x0001, -0x8000], dtype=torch.int16, device="cuda")
    else:
        bits = torch.tensor([0x7F800001, -1, 0x7F800000, -0x00800000, 1, -0x80000000], dtype=torch.int32, device="cuda")
    c["y"] = bits.repeat(M * N // 6 + 1)[:M * N].view(M, N).view(dtype)
    announce(f"lora bits M={M} R={R} {dtype}")
    out = twl.lora_add(**c)
    rows = [t for t in range(M) if t % 3 != 1]
    kind = torch.int16 if dtype == BF else torch.int32
    assert torch.equal(out.view(kind)[rows], c["y"].view(kind)[rows])


def test_python_refusals(twl):
    c = _case(3, 4, 64, 256, 16, 2, F32, [0, 1, 0, 1])
    bad = [dict(y=c["y"].half()), dict(x=c["x"].float()), dict(x=c["x"][:3]), dict(ids=c["ids"].long()), dict(ids=c["ids"][:3]),
           dict(lora_a=c["lora_a"][0]), dict(lora_b=c["lora_b"][:1]), dict(lora_b=c["lora_b"].transpose(1, 2)),
           dict(scale=c["scale"].double()), dict(out=c["y"].bfloat16()), dict(out=c["y"][:2]), dict(out=c["y"].cpu()),
           dict(lora_a=c["lora_a"][:, :12].contiguous(), lora_b=c["lora_b"][..., :12].contiguous())]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, twl.TwlError)):
            twl.lora_add(**{**c, **kw})
    with pytest.raises(twl.TwlError):  # K not a multiple of 128
        twl.lora_add(**{**c, "x": c["x"][:, :120].contiguous(), "lora_a": c["lora_a"][..., :120].contiguous()})
    assert twl.lora_add(**{**c, "y": c["y"][:0], "x": c["x"][:0], "ids": c["ids"][:0]}).shape == (0, 64)
    c = _case(3, 300, 64, 256, 16, 2, F32, runs)  # two kernels: needs a workspace
    assert twl.lora_workspace_bytes(300, 256, 16, 2) > 0
    for ws in (torch.empty(16, dtype=torch.uint8, device="cuda"), c["y"].view(torch.uint8).view(-1)):
        with pytest.raises((ValueError, twl.TwlError)):
            twl.lora_add(workspace=ws, **c)


@pytest.mark.parametrize("M,N,K,R", [(1, 5120, 5120, 16), (3, 260, 17408, 8), (256, 1000, 768, 24), (200, 2048, 8192, 24),
                                     (24, 17408, 5120, 16), (20, 77, 8320, 8), (40, 130, 16384, 16), (1, 1, 128, 8), (1, 70000, 640, 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_launch(twl, M, N, K, R, dtype):
    """Small adapters of up to 256 tokens take one kernel, without a workspace: shares
    of n of more than 1024, rows of A of more than 8192, a last round of few threads;
    in front of a larger buffer, and in place."""
    assert twl.lora_workspace_bytes(M, K, R, 7) == 0
    c = _case(M + N, M, N, K, R, 7, dtype, mixed)
    announce(f"lora one launch M={M} N={N} K={K} R={R} {dtype}")
    buf = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
    _check(twl.lora_add(out=buf[:M], **c), c)
    assert torch.all(buf[M:] == 7.0).item()
    y = c["y"].clone()
    _check(twl.lora_add(**dict(c, out=c["y"])), c, y=y)


# M, N and rank of the two kernels (16 and 64 tokens a tile, each number of rank steps)
TWO_KERNELS = [(20, 72, 32), (80, 1003, 64), (300, 72, 16), (300, 1032, 128)]


@pytest.mark.parametrize("M,N,R", TWO_KERNELS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_stays_with_its_users_two_kernels(twl, M, N, R, dtype):
    """NaN and infinities in one adapter, one token, one row of y and the unused
    adapter reach their own tokens' rows only, through both products' tiles."""
    ids = [t % 4 if t % 7 else -1 for t in range(M)]
    c = _case(M, M, N, 256, R, 5, dtype, ids)
    c["lora_a"][2, 3, 7] = float("nan")
    c["lora_b"][2, :, 1] = float("inf")
    c["lora_a"][4] = float("nan")
    c["lora_b"][4] = float("nan")
    c["x"][5] = float("inf")
    c["y"][9] = float("nan")
    assert twl.lora_workspace_bytes(M, 256, R, 5) > 0
    announce(f"lora nan M={M} N={N} R={R} {dtype}")
    out = twl.lora_add(**c)
    fine = [t for t in range(M) if ids[t] != 2 and t not in (5, 9)]
    c["y"][9] = 0
    out[9] = 0
    with np.errstate(invalid="ignore"):
        _check(out, dict(c, ids=torch.where(torch.arange(M, device="cuda") == 9, 0, c["ids"])), rows=fine)
    assert not torch.isfinite(out[2]).any() and not torch.isfinite(out[5]).all()


@pytest.mark.parametrize("M,N,R", TWO_KERNELS)
def test_rows_and_workspace_behind_the_last_stay(twl, M, N, R):
    c = _case(M, M, N, 256, R, 3, BF, mixed)
    need = twl.lora_workspace_bytes(M, 256, R, 3)
    assert need > 0
    buf = torch.full((M + 3, N), 7.0, dtype=BF, device="cuda")
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    announce(f"lora guards M={M} N={N} R={R}")
    _check(twl.lora_add(out=buf[:M], workspace=ws, **c), c)
    assert torch.all(buf[M:] == 7.0).item()
    assert torch.all(ws[need:] == 0x7F).item()


def test_gradients_are_refused(twl):
    """Adapters that are being trained: no result without a graph; with gradients off
    the same call gives the values."""
    c = _case(2, 5, 64, 256, 16, 2, F32, [0, 1, 0, -1, 1])
    announce("lora grad")
    for name in ("y", "x", "lora_a", "lora_b", "scale"):
        leaf = dict(c, **{name: c[name].detach().clone().requires_grad_()})
        with pytest.raises(ValueError, match=f"{name} requires grad"):
            twl.lora_add(**leaf)
        with torch.no_grad():
            _check(twl.lora_add(**leaf), c)
        with torch.inference_mode():
            _check(twl.lora_add(**leaf), c)
