"""norm_rotate_quant_act on the GPU against the float64 oracle.

h and normed are compared bit for bit: kernel and oracle compute them in fp64
from the same bf16 inputs and round once (through fp32), so they can differ only
where two fp64 values a few 2^-52 apart straddle a rounding border (odds below
1e-9 for an element).  x_i8 and a_scale have to equal rotate_quant_act of the
normed activation bit for bit."""
import numpy as np
import pytest

import oracle.block_oracle as B
import workloads as W
from tests.gpu_helpers import announce, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 1e-6


@pytest.fixture(scope="module")
def twl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_weight_linear_block_amd as m
    m.library()
    return m


def _bits(rng, *shape, scale=1.0, shift=0.0):
    return W.f32_to_bf16_bits((shift + scale * rng.standard_normal(shape)).astype(np.float32))


def _case(seed, M, K, residual, post, gate):
    rng = np.random.default_rng(seed)
    c = {"x_bits": _bits(rng, M, K, scale=0.7), "weight_bits": _bits(rng, K, scale=0.2, shift=1.0),
         "sign": (2 * rng.integers(0, 2, K) - 1).astype(np.int8), "eps": EPS,
         "residual_bits": _bits(rng, M, K, scale=2.0) if residual else None,
         "post_bits": _bits(rng, K, scale=0.2, shift=1.0) if post else None,
         "gate_bits": {"none": None, "channel": _bits(rng, K, shift=0.5), "token": _bits(rng, M, K, shift=0.5)}[gate],
         "branch_scale": 0.75 if residual else 1.0}
    return c


def _t(bits):
    return None if bits is None else dev(bits.view(np.int16))


def _run(twl, c, **kw):
    args = dict(residual=_t(c["residual_bits"]), post_weight=_t(c["post_bits"]), gate=_t(c["gate_bits"]),
                branch_scale=c["branch_scale"], return_normed=True)
    args.update(kw)
    return twl.norm_rotate_quant_act(_t(c["x_bits"]), _t(c["weight_bits"]), None if c["sign"] is None else dev(c["sign"]),
                                     eps=c["eps"], **args)


def _check(got, c, rows=slice(None)):
    x_i8, a_scale, h, normed = got
    ox, oa, oh, on = B.norm_rotate_quant_act(**c)
    assert np.array_equal(host(normed).view(np.uint16)[rows], on[rows]), "normed differs"
    if h is not None:
        assert np.array_equal(host(h).view(np.uint16)[rows], oh[rows]), "h differs"
    if c["sign"] is not None:
        assert np.array_equal(host(x_i8)[rows], ox[rows]), "x_i8 differs"
        assert np.array_equal(host(a_scale).view(np.uint32)[rows], oa.view(np.uint32)[rows]), "a_scale differs"


@pytest.mark.parametrize("residual,post,gate", [
    (False, False, "none"), (True, False, "none"), (True, True, "none"), (True, False, "channel"),
    (True, True, "token"), (False, True, "token"), (False, False, "channel")])
@pytest.mark.parametrize("M,K", [(1, 1024), (3, 5120), (2, 17408)])
def test_forms(twl, M, K, residual, post, gate):
    announce(f"norm M={M} K={K} residual={residual} post={post} gate={gate}")
    c = _case(M * K, M, K, residual, post, gate)
    got = _run(twl, c)
    assert (got[2] is None) == (not residual and not post and gate == "none")
    _check(got, c)


# every number of blocks a wave (1, 2, 4), a last wave with fewer, many tokens
@pytest.mark.parametrize("M,K", [(25, 2048), (2, 16384), (1, 18432), (3, 32768), (2, 33792), (1, 65536), (1500, 1024)])
def test_widths(twl, M, K):
    announce(f"norm M={M} K={K}")
    c = _case(M + K, M, K, True, True, "token")
    _check(_run(twl, c), c)


# more tokens than run at once, in both splits of the row, and three rows a workgroup
@pytest.mark.parametrize("M,K,branch", [
    (800, 2048, False), (1100, 5120, False), (770, 8192, False), (800, 5120, True), (600, 9216, True), (300, 16384, False),
    (300, 16384, True), (1600, 7168, True), (260, 12288, False)])
def test_many_tokens(twl, M, K, branch):
    announce(f"norm M={M} K={K} branch={branch}")
    c = _case(M + K + 1, M, K, branch, branch, "token" if branch else "none")
    _check(_run(twl, c), c)


def test_gate_rows_apart_and_expanded(twl):
    """A gate whose rows lie apart (a slice of a wider tensor), one row expanded,
    and strides that are refused."""
    M, K = 6, 1024
    c = _case(14, M, K, True, True, "token")
    wide = torch.zeros((M, 3 * K + 8), dtype=torch.int16, device="cuda")
    wide[:, K + 8:2 * K + 8] = _t(c["gate_bits"])
    announce("norm gate rows apart")
    _check(_run(twl, c, gate=wide[:, K + 8:2 * K + 8]), c)
    announce("norm gate row expanded")
    one = _t(c["gate_bits"])[:1].expand(M, K)
    _check(_run(twl, c, gate=one), dict(c, gate_bits=np.repeat(c["gate_bits"][:1], M, 0)))
    for bad in (wide[:, :2 * K:2], wide[:, 1:K + 1], torch.zeros((M, K + 4), dtype=torch.int16, device="cuda")[:, :K],
                torch.zeros(M * K, dtype=torch.int16, device="cuda").as_strided((M, K), (8, 1))):
        with pytest.raises((ValueError, twl.TwlError)):
            _run(twl, c, gate=bad)


def test_without_rotation(twl):
    for M, K in ((1, 1024), (700, 2048), (2, 33792)):
        announce(f"norm only M={M} K={K}")
        c = _case(5, M, K, True, False, "none")
        c["sign"] = None
        got = _run(twl, c)
        assert got[0] is None and got[1] is None
        _check(got, c)


def test_extreme_rows(twl):
    """Rows of zeros, of values whose squares overflow fp32, of denormals, a
    single nonzero element; and a row of NaN, which leaves the others alone."""
    K = 2048
    c = _case(11, 6, K, False, True, "none")
    x = W.bf16_bits_to_f32(c["x_bits"]).copy()
    x[0] = 0.0
    x[1] *= 1e30
    x[2] *= 1e-38
    x[3] = 0.0
    x[3, 777] = 3.0
    x[4] = np.nan
    c["x_bits"] = W.f32_to_bf16_bits(np.nan_to_num(x))
    bits = c["x_bits"].copy()
    bits[4] = 0x7FC0
    announce("norm extreme rows")
    got = _run(twl, dict(c, x_bits=bits))
    _check(got, c, rows=[0, 1, 2, 3, 5])
    assert not host(got[0])[0].any() and host(got[1])[0] == 0.0


@pytest.mark.parametrize("weight", [2e-38, 3e-37, 1e-34, 1e-22, 1e-18])
def test_small_weights(twl, weight):
    """Rotated values and scales that are denormal, and either side of the quantiser's
    division."""
    for M, K, branch in ((3, 1024, True), (800, 2048, False)):
        c = _case(17, M, K, branch, branch, "none")
        c["weight_bits"] = W.f32_to_bf16_bits((weight * (1 + 0.2 * np.random.default_rng(3).standard_normal(K))).astype(np.float32))
        announce(f"norm weight={weight} M={M}")
        _check(_run(twl, c), c)


def test_outputs_in_place_and_given(twl):
    c = _case(3, 9, 5120, True, True, "none")
    x, r = _t(c["x_bits"]), _t(c["residual_bits"])
    announce("norm h in place of residual")
    got = _run(twl, c, residual=r, h=r)
    assert got[2] is r
    _check(got, c)
    announce("norm h in place of x, all buffers given")
    out = (torch.empty((9, 5120), dtype=torch.int8, device="cuda"), torch.empty(9, dtype=torch.float32, device="cuda"),
           torch.empty((9, 5120), dtype=torch.bfloat16, device="cuda"))
    x_i8, a_scale, h, normed = twl.norm_rotate_quant_act(
        x, _t(c["weight_bits"]), dev(c["sign"]), eps=EPS, residual=_t(c["residual_bits"]), post_weight=_t(c["post_bits"]),
        branch_scale=c["branch_scale"], x_i8=out[0], a_scale=out[1], normed=out[2], h=x)
    assert x_i8 is out[0] and a_scale is out[1] and normed is out[2] and h is x
    _check((x_i8, a_scale, h, normed.view(torch.int16)), c)


def test_rows_behind_the_last_stay(twl):
    """Outputs in the front of larger buffers: what lies behind is left."""
    M, K = 5, 1024
    c = _case(8, M, K, True, False, "none")
    bufs = [torch.full((M + 2, K), 77, dtype=torch.int8, device="cuda"), torch.full((M + 8,), 7.0, device="cuda"),
            torch.full((M + 2, K), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((M + 2, K), 7.0, dtype=torch.bfloat16, device="cuda")]
    announce("norm guard rows")
    x_i8, a_scale, h, normed = _run(twl, c, x_i8=bufs[0][:M], a_scale=bufs[1][:M], h=bufs[2][:M], normed=bufs[3][:M])
    _check((x_i8, a_scale, h.view(torch.int16), normed.view(torch.int16)), c)
    for b, v in zip(bufs, (77, 7, 7, 7)):
        assert torch.all(b[M:].float() == v).item()


def test_other_stream_and_graph(twl):
    """On a stream of its own, and captured: replays follow changed inputs."""
    c = _case(21, 24, 5120, True, True, "channel")
    x, w, sign = _t(c["x_bits"]), _t(c["weight_bits"]), dev(c["sign"])
    res, post, gate = _t(c["residual_bits"]), _t(c["post_bits"]), _t(c["gate_bits"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    announce("norm on another stream")
    got = twl.norm_rotate_quant_act(x, w, sign, eps=EPS, residual=res, post_weight=post, gate=gate,
                                    branch_scale=c["branch_scale"], return_normed=True, stream=s)
    s.synchronize()
    _check(got, c)
    announce("norm captured")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = twl.norm_rotate_quant_act(x, w, sign, eps=EPS, residual=res, post_weight=post, gate=gate,
                                        branch_scale=c["branch_scale"], return_normed=True)
    for k in range(3):
        c2 = _case(30 + k, 24, 5120, True, True, "channel")
        for t, name in ((x, "x_bits"), (res, "residual_bits")):
            t.copy_(_t(c2[name]))
        g.replay()
        torch.cuda.synchronize()
        _check(got, dict(c, x_bits=c2["x_bits"], residual_bits=c2["residual_bits"]))


def test_python_refusals(twl):
    x = torch.zeros((4, 1024), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1024, dtype=torch.bfloat16, device="cuda")
    sign = torch.ones(1024, dtype=torch.int8, device="cuda")
    f = twl.norm_rotate_quant_act
    for bad in (dict(residual=x[:3]), dict(post_weight=w[:512]), dict(gate=x[:2]), dict(x_i8=torch.empty_like(x)[:1]),
                dict(residual=torch.zeros((1024, 4), dtype=torch.bfloat16, device="cuda").t()), dict(normed=x),
                dict(residual=x.cpu()), dict(h=x)):
        with pytest.raises((ValueError, TypeError, twl.TwlError)):
            f(x, w, sign, **bad)
    with pytest.raises(TypeError):
        f(x.float(), w, sign)
    with pytest.raises(ValueError):
        f(x[0], w, sign)
    with pytest.raises(twl.TwlError):
        f(x, w, sign, eps=0.0)
    with pytest.raises(twl.TwlError):
        f(x, w, None)
    out = f(x[:0], w, sign)
    assert out[0].shape == (0, 1024)


# exponents of x, post_weight, gate, branch_scale, residual and weight (None: not
# there); products of some of them leave fp32's range on either side, h and n do not
@pytest.mark.parametrize("x,post,gate,scale,residual,weight", [
    (100, None, 40, -60, None, 0),     # x * gate above 2^128
    (100, None, 40, -60, 79, 0),
    (60, 100, 60, -120, None, 0),      # x * post_weight, and times gate
    (120, 100, 20, -90, 29, 0),        # the same of a row whose squares pass fp32's range
    (-100, None, -60, 150, None, 0),   # x * gate below 2^-149
    (-60, -70, -60, 130, 0, 0),
    (60, None, None, 0, 60, 100),      # h * weight above 2^128
    (-60, None, None, 0, -60, -110),   # and below 2^-149: n is 2^-110
    (11, None, None, 0, 11, 112),      # the largest and smallest rows that are not scaled
    (-7, None, None, 0, -7, -117),
])
@pytest.mark.parametrize("M,K,gate_rows", [(3, 1024, True), (2, 17408, False), (1, 33792, True)])
def test_products_outside_fp32(twl, M, K, gate_rows, x, post, gate, scale, residual, weight):
    c = _case(41, M, K, residual is not None, post is not None,
              "none" if gate is None else "token" if gate_rows else "channel")
    c["branch_scale"], c["eps"] = 2.0 ** scale, 1e-40
    for name, e in (("x_bits", x), ("post_bits", post), ("gate_bits", gate), ("residual_bits", residual), ("weight_bits", weight)):
        if e is not None:
            c[name] = W.f32_to_bf16_bits((W.bf16_bits_to_f32(c[name]).astype(np.float64) * 2.0 ** e).astype(np.float32))
    _, oa, oh, on = B.norm_rotate_quant_act(**c)
    for bits in (oh, on):  # what is defined is finite and not flushed
        v = W.bf16_bits_to_f32(bits)
        assert np.isfinite(v).all() and np.abs(v).max() > 2.0 ** -120
    announce(f"norm products M={M} K={K} x={x} post={post} gate={gate} scale={scale} residual={residual} weight={weight}")
    _check(_run(twl, c), c)


@pytest.mark.parametrize("M,K", [(800, 2048), (3, 2048)])
@pytest.mark.parametrize("x,weight", [(60, 100), (-60, -80)])
def test_products_outside_fp32_of_the_norm_alone(twl, M, K, x, weight):
    """h is x itself; the second of two tokens of a workgroup too."""
    c = _case(43, M, K, False, False, "none")
    c["eps"] = 1e-40
    for name, e in (("x_bits", x), ("weight_bits", weight)):
        c[name] = W.f32_to_bf16_bits(W.bf16_bits_to_f32(c[name]) * np.float32(2.0 ** e))
    announce(f"norm alone, products M={M} x={x} weight={weight}")
    _check(_run(twl, c), c)


def test_gradients_are_refused(twl):
    c = _case(51, 3, 1024, True, True, "channel")
    bf = {k: _t(c[k]).view(torch.bfloat16).requires_grad_() for k in ("x_bits", "weight_bits", "residual_bits", "post_bits", "gate_bits")}
    announce("norm grad")

    def run(**kw):
        t = {k: v.detach() for k, v in bf.items()}
        t.update(kw)
        return twl.norm_rotate_quant_act(t["x_bits"], t["weight_bits"], dev(c["sign"]), eps=EPS, residual=t["residual_bits"],
                                         post_weight=t["post_bits"], gate=t["gate_bits"], branch_scale=c["branch_scale"],
                                         return_normed=True)

    for k, v in bf.items():
        with pytest.raises(ValueError, match="requires grad"):
            run(**{k: v})
    with torch.no_grad():
        x_i8, a_scale, h, normed = run(**bf)
    _check((x_i8, a_scale, h.view(torch.int16), normed.view(torch.int16)), c)
