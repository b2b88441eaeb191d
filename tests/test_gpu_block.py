"""The block operators together, as a served feed-forward block with adapters runs
them: norm_rotate_quant_act -> ternary_gated_linear -> rotate_quant_act ->
ternary_linear -> lora_add -> norm_rotate_quant_act.  Every step is checked against
the oracle on the step's own GPU inputs, so a wrong hand-over shows where it
happens, and a captured graph of the whole has to give the eager run's bits.  Also
sizes whose offsets pass 32 bits."""
import numpy as np
import pytest

import oracle.block_oracle as B
import oracle.twl_oracle as O
import workloads as W
from tests.gpu_helpers import announce, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def twl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_weight_linear_block_amd as m
    m.library()
    return m


def _bits(t):
    return host(t.view(torch.int16)).view(np.uint16)


def _model(twl, H, I, R, n, seed):
    """Weights of one block: hidden width H, intermediate width I, n adapters of rank R."""
    rng = np.random.default_rng(seed)
    gate, up, down = (W.make_layer(seed + k, 1, K, N) for k, (K, N) in enumerate(((H, I), (H, I), (I, H))))
    bf = lambda *s, c=1.0, m=0.0: dev(W.f32_to_bf16_bits((m + c * rng.standard_normal(s)).astype(np.float32)).view(np.int16)).view(torch.bfloat16)  # noqa: E731
    return dict(
        host=(gate, up, down),
        gated=twl.pack_ternary_gated(dev(gate.code), dev(gate.s_bits.view(np.int16)), dev(up.code), dev(up.s_bits.view(np.int16))),
        down=twl.pack_ternary(dev(down.code), dev(down.s_bits.view(np.int16))),
        sign_h=dev(gate.sign), sign_i=dev(down.sign), w1=bf(H, c=0.2, m=1.0), w2=bf(H, c=0.2, m=1.0), post=bf(H, c=0.2, m=1.0),
        lora_a=bf(n, R, I, c=I ** -0.5), lora_b=bf(n, H, R, c=0.3), scale=dev(rng.uniform(0.5, 2, n).astype(np.float32)))


def _block(twl, m, x, residual, ids):
    """One block; every intermediate result, by name."""
    r = {}
    r["x1"], r["s1"], r["h1"], _ = twl.norm_rotate_quant_act(x, m["w1"], m["sign_h"], eps=EPS, residual=residual)
    r["act"] = twl.ternary_gated_linear(r["x1"], r["s1"], *m["gated"])
    r["x2"], r["s2"] = twl.rotate_quant_act(r["act"], m["sign_i"])
    r["y"] = twl.ternary_linear_bf16(r["x2"], r["s2"], *m["down"])
    r["ya"] = twl.lora_add(r["y"], r["act"], ids, m["lora_a"], m["lora_b"], m["scale"])
    r["x3"], r["s3"], r["h2"], r["n2"] = twl.norm_rotate_quant_act(
        r["ya"], m["w2"], m["sign_h"], eps=EPS, residual=r["h1"], post_weight=m["post"], branch_scale=0.5, return_normed=True)
    return r


def _check_block(m, x, residual, ids, r):
    gate, up, down = m["host"]
    sign_h, sign_i = host(m["sign_h"]), host(m["sign_i"])
    ox, os_, oh, _ = B.norm_rotate_quant_act(_bits(x), _bits(m["w1"]), sign_h, EPS, residual_bits=_bits(residual))
    assert np.array_equal(host(r["x1"]), ox) and np.array_equal(host(r["s1"]), os_) and np.array_equal(_bits(r["h1"]), oh)
    _, qg, sg = O.pack_ternary(gate.code, gate.s_bits)
    _, qu, su = O.pack_ternary(up.code, up.s_bits)
    want, mag, mag_u = B.gated_linear(ox, os_, gate.code, qg, sg, up.code, qu, su)
    got = host(r["act"].float()).astype(np.float64)
    # the bounds of test_gpu_gated.py and test_gpu_lora.py
    assert np.all(np.abs(got - want) <= np.abs(want) * ((5 * mag + 16) * U + 2.0 ** -8) + 2.0 ** -126 * (1 + mag * mag_u))
    ox, os_ = O.rotate_quant_act(_bits(r["act"]), sign_i)
    assert np.array_equal(host(r["x2"]), ox) and np.array_equal(host(r["s2"]), os_)
    _, qd, sd = O.pack_ternary(down.code, down.s_bits)
    y = O.epilogue(O.linear_acc(ox, down.code, qd), os_, sd).astype(np.float64)
    got = host(r["y"].float()).astype(np.float64)
    assert np.all(np.abs(got - y) <= np.abs(y) * (2.0 ** -8 + 8 * U))
    f = lambda t: host(t.float()).astype(np.float64)  # noqa: E731
    want, mag_x, mag_v = B.lora_add(f(r["y"]), f(r["act"]), host(ids), f(m["lora_a"]), f(m["lora_b"]), host(m["scale"]))
    K, R = r["act"].shape[1], m["lora_a"].shape[1]
    delta = (K + 64) * U * mag_x + (2.0 ** -16 + (3 * R + 8) * U) * mag_v
    assert np.all(np.abs(f(r["ya"]) - want) <= delta + (np.abs(want) + delta) * (2.0 ** -8 + U))
    ox, os_, oh, on = B.norm_rotate_quant_act(_bits(r["ya"]), _bits(m["w2"]), sign_h, EPS, residual_bits=oh,
                                              post_bits=_bits(m["post"]), branch_scale=0.5)
    assert np.array_equal(host(r["x3"]), ox) and np.array_equal(host(r["s3"]), os_)
    assert np.array_equal(_bits(r["h2"]), oh) and np.array_equal(_bits(r["n2"]), on)


@pytest.mark.parametrize("M,H,I", [(1, 1024, 5120), (24, 2048, 4096), (130, 1024, 2048)])
def test_block_eager_and_captured(twl, M, H, I):
    m = _model(twl, H, I, 16, 5, 3)
    rng = np.random.default_rng(M)

    def inputs():
        t = lambda c: torch.from_numpy((c * rng.standard_normal((M, H))).astype(np.float32)).cuda().bfloat16()  # noqa: E731
        return t(0.5), t(2.0), torch.from_numpy(rng.integers(-1, 5, M).astype(np.int32)).cuda()

    announce(f"block M={M} H={H} I={I}")
    x, residual, ids = inputs()
    _check_block(m, x, residual, ids, _block(twl, m, x, residual, ids))
    announce(f"block captured M={M} H={H} I={I}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the linear layer keeps its workspace by stream: made before the capture
        _block(twl, m, x, residual, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept = _block(twl, m, x, residual, ids)
    for _ in range(3):
        for t, new in zip((x, residual, ids), inputs()):
            t.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = _block(twl, m, x, residual, ids)
        for name in eager:
            assert torch.equal(kept[name], eager[name]), name
    _check_block(m, x, residual, ids, eager)


def test_norm_rows_past_32_bits(twl):
    """2^31 elements and some: rows at the start, the middle and the end."""
    M, K = 65600, 32768
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 32767, 32768, 65535, 65536, M - 1]
    rng = np.random.default_rng(5)
    bits = W.f32_to_bf16_bits(rng.standard_normal((len(rows), K)).astype(np.float32))
    x[rows] = dev(bits.view(np.int16)).view(torch.bfloat16)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    sign = dev((2 * rng.integers(0, 2, K) - 1).astype(np.int8))
    announce("norm 65600 x 32768")
    x_i8, a_scale, h, normed = twl.norm_rotate_quant_act(x, w, sign, eps=EPS, branch_scale=0.5, return_normed=True)
    ox, oa, oh, on = B.norm_rotate_quant_act(bits, _bits(w), host(sign), EPS, branch_scale=0.5)
    at = torch.tensor(rows, device="cuda")
    assert np.array_equal(host(x_i8[at]), ox) and np.array_equal(host(a_scale[at]), oa)
    assert np.array_equal(_bits(h[at]), oh) and np.array_equal(_bits(normed[at]), on)
    assert int((a_scale != 0).sum()) == len(rows)


def test_lora_rows_past_32_bits(twl):
    M, N, K, R, n = 66000, 32776, 128, 8, 3
    rows = [0, 70, 32767, 65521, 65536, 65999]
    g = torch.Generator(device="cuda").manual_seed(3)
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[rows] = torch.tensor([0, 1, 2, 1, 0, 2], dtype=torch.int32, device="cuda")
    a = torch.randn((n, R, K), generator=g, device="cuda").bfloat16()
    b = torch.randn((n, N, R), generator=g, device="cuda").bfloat16()
    scale = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    announce("lora 66000 x 32776")
    out = twl.lora_add(y, x, ids, a, b, scale, out=y)
    f = lambda t: host(t.float()).astype(np.float64)  # noqa: E731
    want, mag_x, mag_v = B.lora_add(np.zeros((len(rows), N)), f(x[rows]), host(ids[rows]), f(a), f(b), host(scale))
    delta = (K + 64) * U * mag_x + (2.0 ** -16 + (3 * R + 8) * U) * mag_v
    assert np.all(np.abs(f(out[rows]) - want) <= delta + (np.abs(want) + delta) * (2.0 ** -8 + U))
    out[rows] = 0
    assert not out.any().item()
