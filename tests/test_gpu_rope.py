"""qk_norm_rope on the GPU against the float64 oracle, element by element.

The bound.  u = 2^-24.  The sum of D squares in fp32 is off by at most the roundings of a
chain: 8 in a lane and up to 5 exchanges, 13 u; the mean and eps add 2 u, half of that passes
the reciprocal root, which adds 2 u (1 ulp): n = x r w is within 15/2 + 2 + 2 < 13 u of
its value.  A turned element adds two products: within (13 + 2) u of |a c| + |b s|.  One
rounding to bf16: 2^-8 of the result.  Products below bf16's smallest normal number round by
at most 2^-134."""
import numpy as np
import pytest

import oracle.attention_oracle as A
from tests.gpu_helpers import announce, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TINY = 2.0 ** -134


@pytest.fixture(scope="module")
def twl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_weight_linear_block_amd as m
    m.library()
    return m


def _table(n_pos, rot, base=1e6):
    ang = np.arange(n_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _case(seed, M, n_q, n_kv, D, rot, dtype=torch.bfloat16, norm=True, n_pos=500, page=16, scale=1.0):
    rng = np.random.default_rng(seed)
    pages = M // page + 4
    slots = rng.permutation(pages * page)[:M].astype(np.int32)
    c = dict(qkv=(torch.from_numpy(rng.standard_normal((M, (n_q + 2 * n_kv) * D)).astype(np.float32)) * scale).to(dtype).cuda(),
             positions=dev(rng.integers(0, n_pos, M).astype(np.int32)) if rot else None, cos_sin=dev(_table(n_pos, rot)) if rot else None,
             slots=dev(slots))
    for n in ("q_weight", "k_weight"):
        c[n] = torch.from_numpy(1 + 0.3 * rng.standard_normal(D).astype(np.float32)).bfloat16().cuda() if norm else None
    for n in ("k_cache", "v_cache"):
        c[n] = torch.from_numpy(rng.standard_normal((pages, n_kv, page, D)).astype(np.float32)).bfloat16().cuda()
    return c


def _np(t):
    return host(t.float()).astype(np.float64)


def _want(c, n_q, n_kv, eps=1e-6, interleaved=False):
    x = _np(c["qkv"])
    M, D = x.shape[0], x.shape[1] // (n_q + 2 * n_kv)
    x = x.reshape(M, -1, D)
    if c["cos_sin"] is None:
        cos = sin = np.zeros((M, 0))
    else:
        t = host(c["cos_sin"])[np.clip(host(c["positions"]), 0, c["cos_sin"].shape[0] - 1)]
        cos, sin = np.split(t, 2, 1)
    out = [A.heads_norm_rope(x[:, :n_q], None if c["q_weight"] is None else _np(c["q_weight"]), eps, cos, sin, interleaved),
           A.heads_norm_rope(x[:, n_q:n_q + n_kv], None if c["k_weight"] is None else _np(c["k_weight"]), eps, cos, sin, interleaved)]
    return out[0], out[1], x[:, n_q + n_kv:]


def _near(got, want, mag):
    tol = 15 * U * mag
    tol = tol + (np.abs(want) + tol) * 2.0 ** -8 + TINY
    err = np.abs(got - want)
    assert (err <= tol).all(), float(np.max(err / tol))


def _check(c, out, before, n_q, n_kv, written=None, stored=None, interleaved=False, eps=1e-6):
    """Queries of the `written` tokens, cache slots of the `stored` ones; all other slots as before."""
    q, k_cache, v_cache = out
    (wq, mq), (wk, mk), wv = _want(c, n_q, n_kv, eps, interleaved)
    M = wq.shape[0]
    written = np.ones(M, bool) if written is None else written
    stored = written if stored is None else stored
    _near(_np(q)[written], wq[written], mq[written])
    page = k_cache.shape[2]
    slots = host(c["slots"])[stored]
    for cache, old, want, mag in ((k_cache, before[0], wk, mk), (v_cache, before[1], wv, np.abs(wv) * 0)):
        got = _np(cache)
        _near(got[slots // page, :, slots % page], want[stored], mag[stored])
        old = _np(old)
        old[slots // page, :, slots % page] = got[slots // page, :, slots % page]
        assert np.array_equal(got, old)


def _run(twl, c, n_q, n_kv, **kw):
    before = c["k_cache"].clone(), c["v_cache"].clone()
    out = twl.qk_norm_rope(c["qkv"], c["positions"], c["cos_sin"], n_q, n_kv, q_weight=c["q_weight"], k_weight=c["k_weight"],
                           slots=c["slots"], k_cache=c["k_cache"], v_cache=c["v_cache"], **kw)
    assert out[1] is c["k_cache"] and out[2] is c["v_cache"]
    return out, before


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("D,n_q,n_kv,rot", [(64, 1, 1, 64), (64, 9, 3, 32), (64, 16, 2, 16), (128, 40, 8, 128), (128, 5, 1, 64), (128, 3, 3, 32),
                                            (128, 6, 2, 48), (256, 20, 4, 64), (256, 7, 7, 256), (256, 1, 1, 208), (64, 5, 5, 48)])
@pytest.mark.parametrize("M", [1, 3, 37])
def test_values(twl, M, D, n_q, n_kv, rot, dtype):
    announce(f"qk_norm_rope {M} tokens {n_q}/{n_kv} x {D} rot {rot} {dtype}")
    for interleaved in (False, True):
        c = _case(M * D + rot, M, n_q, n_kv, D, rot, dtype)
        out, before = _run(twl, c, n_q, n_kv, interleaved=interleaved)
        _check(c, out, before, n_q, n_kv, interleaved=interleaved)


@pytest.mark.parametrize("M", [300, 2100])
@pytest.mark.parametrize("D,n_q,n_kv,rot", [(64, 16, 2, 64), (128, 40, 8, 128), (256, 20, 4, 64)])
def test_many_tokens(twl, M, D, n_q, n_kv, rot):
    c = _case(M, M, n_q, n_kv, D, rot, page=64)
    out, before = _run(twl, c, n_q, n_kv)
    _check(c, out, before, n_q, n_kv)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("which", ["none", "q", "k", "no rotation"])
def test_parts_left_out(twl, D, which):
    c = _case(D, 9, 4, 2, D, 0 if which == "no rotation" else 32)
    if which in ("none", "k"):
        c["q_weight"] = None
    if which in ("none", "q"):
        c["k_weight"] = None
    out, before = _run(twl, c, 4, 2)
    _check(c, out, before, 4, 2)


def test_without_caches(twl):
    c = _case(3, 21, 6, 2, 128, 128)
    q, k, v = twl.qk_norm_rope(c["qkv"], c["positions"], c["cos_sin"], 6, 2, q_weight=c["q_weight"], k_weight=c["k_weight"])
    out, _ = _run(twl, c, 6, 2)
    assert torch.equal(q, out[0]) and k.shape == v.shape == (21, 2, 128)
    page, at = c["slots"].long() // 16, c["slots"].long() % 16
    assert torch.equal(k, c["k_cache"][page, :, at]) and torch.equal(v, c["v_cache"][page, :, at])


@pytest.mark.parametrize("page", [1, 2, 8, 1024])
def test_page_sizes(twl, page):
    c = _case(4, 50, 4, 2, 64, 64, page=page)
    out, before = _run(twl, c, 4, 2)
    _check(c, out, before, 4, 2)


@pytest.mark.parametrize("M", [40, 900])
def test_padding(twl, M):
    c = _case(5, M, 8, 2, 128, 64)
    pos, slots = host(c["positions"]).copy(), host(c["slots"]).copy()
    pos[::5], pos[1::7] = -1, 500
    slots[2::3] = -1
    slots[7] = c["k_cache"].shape[0] * 16
    slots[8] = 2 ** 31 - 1
    c["positions"], c["slots"] = dev(pos), dev(slots)
    q = torch.full((M, 8, 128), 3.0, device="cuda").bfloat16()
    out, before = _run(twl, c, 8, 2, q=q)
    written = (pos >= 0) & (pos < 500)
    stored = written & (slots >= 0) & (slots < c["k_cache"].shape[0] * 16)
    _check(c, out, before, 8, 2, written=written, stored=stored)
    assert (q[torch.from_numpy(~written).cuda()] == 3).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_rows_apart(twl, dtype):
    c = _case(6, 30, 6, 2, 64, 64, dtype)
    wide = torch.full((30, 10 * 64 + 24), float("nan"), device="cuda").to(dtype)
    wide[:, 16:16 + 640] = c["qkv"]
    dense = twl.qk_norm_rope(c["qkv"], c["positions"], c["cos_sin"], 6, 2, q_weight=c["q_weight"])
    apart = twl.qk_norm_rope(wide[:, 16:16 + 640], c["positions"], c["cos_sin"], 6, 2, q_weight=c["q_weight"])
    for a, b in zip(dense, apart):
        assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [0.0, 1e-4, 300.0])
def test_sizes_of_values(twl, scale):
    c = _case(7, 11, 4, 2, 128, 128, torch.float32, scale=scale)
    out, before = _run(twl, c, 4, 2, eps=1e-5)
    _check(c, out, before, 4, 2, eps=1e-5)


def test_not_finite_stays_in_its_head(twl):
    for bad in (float("nan"), float("inf")):
        c = _case(8, 6, 4, 2, 64, 64)
        clean, _ = _run(twl, c, 4, 2)
        clean = [t.clone() for t in clean]
        c["qkv"][2, 64 + 5] = bad       # query head 1 of token 2
        c["qkv"][3, 4 * 64 + 1] = bad   # key head 0 of token 3
        c["qkv"][4, 7 * 64 + 9] = bad   # value head 1 of token 4
        out, _ = _run(twl, c, 4, 2)
        slots, page = host(c["slots"]), 16
        hit = torch.zeros_like(out[0], dtype=torch.bool)
        hit[2, 1] = True
        assert torch.equal(out[0][~hit], clean[0][~hit]) and not torch.isfinite(out[0][2, 1, 5])
        hit = torch.zeros_like(out[1], dtype=torch.bool)
        hit[slots[3] // page, 0, slots[3] % page] = True
        assert torch.equal(out[1][~hit], clean[1][~hit]) and not torch.isfinite(out[1][slots[3] // page, 0, slots[3] % page, 1])
        hit = torch.zeros_like(out[2], dtype=torch.bool)
        hit[slots[4] // page, 1, slots[4] % page, 9] = True
        assert torch.equal(out[2][~hit], clean[2][~hit]) and not torch.isfinite(out[2][hit]).any()


def test_cache_past_32_bit_offsets(twl):
    """A cache of 2^31 elements and more: the first and the last slots."""
    pages = 2 ** 31 // (8 * 64 * 128) + 3
    c = _case(9, 4, 8, 8, 128, 128)
    c["k_cache"] = torch.zeros((pages, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
    c["v_cache"] = torch.zeros((pages, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
    c["slots"] = dev(np.array([0, pages * 64 - 1, (pages - 2) * 64 + 5, 77], np.int32))
    twl.qk_norm_rope(c["qkv"], c["positions"], c["cos_sin"], 8, 8, slots=c["slots"], k_cache=c["k_cache"], v_cache=c["v_cache"])
    q, k, v = twl.qk_norm_rope(c["qkv"], c["positions"], c["cos_sin"], 8, 8)
    page, at = c["slots"].long() // 64, c["slots"].long() % 64
    assert torch.equal(c["k_cache"][page, :, at], k) and torch.equal(c["v_cache"][page, :, at], v)
    assert int(torch.count_nonzero(c["v_cache"][page.min():page.max() + 1].view(torch.int16)[1:2])) == int(
        torch.count_nonzero(v[3].view(torch.int16)))


def test_stream_and_graph(twl):
    c = _case(10, 24, 8, 2, 128, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, before = _run(twl, c, 8, 2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(c, out, before, 8, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = twl.qk_norm_rope(c["qkv"], c["positions"], c["cos_sin"], 8, 2, slots=c["slots"], k_cache=c["k_cache"], v_cache=c["v_cache"])
    for r in range(3):
        c["qkv"].copy_(torch.roll(c["qkv"], 1, 0))
        c["positions"].add_(1)
        c["slots"].copy_(torch.roll(c["slots"], 5, 0))
        eager = twl.qk_norm_rope(c["qkv"], c["positions"], c["cos_sin"], 8, 2, slots=c["slots"], k_cache=before[0], v_cache=before[1])
        graph.replay()
        torch.cuda.synchronize()
        page, at = c["slots"].long() // 16, c["slots"].long() % 16
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1][page, :, at], before[0][page, :, at])
        assert torch.equal(got[2][page, :, at], before[1][page, :, at])


def test_empty_and_refusals(twl):
    c = _case(11, 4, 4, 2, 64, 64)
    q, k, v = twl.qk_norm_rope(c["qkv"][:0], c["positions"][:0], c["cos_sin"], 4, 2)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    call = lambda **kw: twl.qk_norm_rope(kw.pop("qkv", c["qkv"]), kw.pop("positions", c["positions"]), kw.pop("cos_sin", c["cos_sin"]),  # noqa: E731
                                         kw.pop("n_q", 4), kw.pop("n_kv", 2), **kw)
    for kw, error, word in [(dict(n_q=3), ValueError, "columns"), (dict(n_q=0), ValueError, "n_q"), (dict(cos_sin=None), ValueError, "cos_sin"),
                            (dict(positions=c["positions"][:3]), ValueError, "positions"), (dict(slots=c["slots"]), ValueError, "slots"),
                            (dict(k_cache=c["k_cache"], slots=c["slots"]), ValueError, "together"),
                            (dict(q_weight=c["q_weight"][:32].contiguous()), ValueError, "q_weight"),
                            (dict(qkv=c["qkv"].half()), TypeError, "qkv"), (dict(qkv=c["qkv"].clone().requires_grad_()), ValueError, "requires grad"),
                            (dict(positions=c["positions"].long()), TypeError, "positions"),
                            (dict(cos_sin=c["cos_sin"][:, :24].contiguous()), twl.TwlError, "rot"),
                            (dict(k_cache=c["k_cache"][:, :1].contiguous(), v_cache=c["v_cache"][:, :1].contiguous(), slots=c["slots"]), ValueError, "k_cache"),
                            (dict(k_cache=c["k_cache"], v_cache=c["k_cache"], slots=c["slots"]), twl.TwlError, "overlaps"),
                            (dict(eps=0.0), twl.TwlError, "eps")]:
        with pytest.raises(error, match=word):
            call(**kw)
    with pytest.raises(twl.TwlError, match="head size"):
        twl.qk_norm_rope(torch.zeros((2, 3 * 32), device="cuda"), None, None, 1, 1)
