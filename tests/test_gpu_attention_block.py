"""The operators of a block's attention half together, as a server runs them over batches of
prompts, chunks and single tokens: norm_rotate_quant_act -> ternary_linear (queries, keys,
values) -> qk_norm_rope -> window_attention -> rotate_quant_act -> int8_linear (the output
projection).  Every step is checked against the oracle on the step's own GPU inputs, the cache
against what earlier batches left in it, and a captured graph of the whole, replayed for
growing sequences, has to give the eager run's bits."""
import numpy as np
import pytest

import oracle.attention_oracle as A
import oracle.block_oracle as B
import oracle.twl_oracle as O
import workloads as W
from tests import test_gpu_attention, test_gpu_int8, test_gpu_rope
from tests.gpu_helpers import announce, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 1e-6
N_POS = 400


@pytest.fixture(scope="module")
def twl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_weight_linear_block_amd as m
    m.library()
    return m


def _bits(t):
    return host(t.view(torch.int16)).view(np.uint16)


def _model(twl, H, n_q, n_kv, D, page, pages, seed):
    rng = np.random.default_rng(seed)
    qkv = W.make_layer(seed, 1, H, (n_q + 2 * n_kv) * D)
    bf = lambda *s, c=0.2, m=1.0: torch.from_numpy((m + c * rng.standard_normal(s)).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    sign_o = dev((2 * rng.integers(0, 2, n_q * D) - 1).astype(np.int8))
    m = dict(host=qkv, qkv=twl.pack_ternary(dev(qkv.code), dev(qkv.s_bits.view(np.int16))), sign_h=dev(qkv.sign), sign_o=sign_o,
             w=bf(H), q_weight=bf(D), k_weight=bf(D), n_q=n_q, n_kv=n_kv, D=D, page=page, cos_sin=dev(test_gpu_rope._table(N_POS, D)))
    m["o"] = twl.rotate_quant_act(bf(H, n_q * D, c=(n_q * D) ** -0.5, m=0.0), sign_o)
    for n in ("k_cache", "v_cache"):
        m[n] = bf(pages, n_kv, page, D)
    return m


def _half(twl, m, x, residual, positions, slots, table, q_start, kv_len, window, sinks):
    """One attention half; every intermediate result, by name."""
    r = {}
    r["x1"], r["s1"], r["h"], _ = twl.norm_rotate_quant_act(x, m["w"], m["sign_h"], eps=EPS, residual=residual)
    r["qkv"] = twl.ternary_linear_bf16(r["x1"], r["s1"], *m["qkv"])
    r["q"] = torch.zeros((x.shape[0], m["n_q"], m["D"]), dtype=torch.bfloat16, device="cuda")  # padding's rows: no kernel writes them
    twl.qk_norm_rope(r["qkv"], positions, m["cos_sin"], m["n_q"], m["n_kv"], q_weight=m["q_weight"], k_weight=m["k_weight"], eps=EPS,
                     slots=slots, k_cache=m["k_cache"], v_cache=m["v_cache"], q=r["q"])
    r["o"] = torch.zeros_like(r["q"])
    twl.window_attention(r["q"], m["k_cache"], m["v_cache"], table, q_start, kv_len, window=window, sinks=sinks, out=r["o"])
    r["x2"], r["s2"] = twl.rotate_quant_act(r["o"].view(x.shape[0], -1), m["sign_o"])
    r["y"] = twl.int8_linear(r["x2"], r["s2"], *m["o"], out_dtype=torch.bfloat16)
    return r


def _check(m, before, x, residual, step, window, sinks, r):
    ox, os_, oh, _ = B.norm_rotate_quant_act(_bits(x), _bits(m["w"]), host(m["sign_h"]), EPS, residual_bits=_bits(residual))
    assert np.array_equal(host(r["x1"]), ox) and np.array_equal(host(r["s1"]), os_) and np.array_equal(_bits(r["h"]), oh)
    layer = m["host"]
    _, g, s = O.pack_ternary(layer.code, layer.s_bits)
    want = O.epilogue(O.linear_acc(ox, layer.code, g), os_, s).astype(np.float64)
    got = host(r["qkv"].float()).astype(np.float64)
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 8 * 2.0 ** -24))
    positions, slots, table, q_start, kv_len = step
    real = host(positions) >= 0
    c = dict(qkv=r["qkv"], positions=positions, cos_sin=m["cos_sin"], slots=slots, q_weight=m["q_weight"], k_weight=m["k_weight"])
    test_gpu_rope._check(c, (r["q"], m["k_cache"], m["v_cache"]), before, m["n_q"], m["n_kv"], written=real)
    assert (r["q"][torch.from_numpy(~real).cuda()] == 0).all()
    c = dict(q=r["q"], k_cache=m["k_cache"], v_cache=m["v_cache"], page_table=table, q_start=q_start, kv_len=kv_len)
    test_gpu_attention._check(c, r["o"], window=window, sinks=sinks)
    ox, os_ = O.rotate_quant_act(_bits(r["o"].view(x.shape[0], -1)), host(m["sign_o"]))
    assert np.array_equal(host(r["x2"]), ox) and np.array_equal(host(r["s2"]), os_)
    _, want, mag = A.int8_linear(ox, os_, host(m["o"][0]), host(m["o"][1]))
    test_gpu_int8._compare(r["y"], want, mag, torch.bfloat16)


class Server:
    """Sequences over pages: the host's side of a batch."""

    def __init__(self, m, sequences, seed):
        self.m, self.rng, self.len = m, np.random.default_rng(seed), np.zeros(sequences, np.int64)
        pages = m["k_cache"].shape[0]
        self.table = self.rng.permutation(pages)[:pages // sequences * sequences].reshape(sequences, -1).astype(np.int32)

    def step(self, lengths, M):
        """positions, slots, table, q_start, kv_len of a batch of M rows, those behind the sequences' padding."""
        positions, slots = np.full(M, -1, np.int32), np.full(M, -1, np.int32)
        at, page = 0, self.m["page"]
        for b, n in enumerate(lengths):
            p = self.len[b] + np.arange(n)
            positions[at:at + n], slots[at:at + n] = p, self.table[b, p // page] * page + p % page
            at, self.len[b] = at + n, self.len[b] + n
        starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        return [positions, slots, self.table, starts, self.len.astype(np.int32)]

    def rows(self, M, H):
        return [torch.from_numpy(self.rng.standard_normal((M, H)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]


@pytest.mark.parametrize("H,n_q,n_kv,D,page,window,sinks", [(1024, 8, 2, 128, 16, 0, 0), (2048, 16, 4, 64, 32, 40, 4), (1024, 4, 1, 256, 64, 100, 0)])
def test_eager_and_captured(twl, H, n_q, n_kv, D, page, window, sinks):
    m = _model(twl, H, n_q, n_kv, D, page, 3 * (N_POS // page), 3)
    server = Server(m, 3, 4)
    for lengths, M in (([50, 7, 133], 200), ([1, 60, 1], 62), ([4, 0, 3], 8)):
        announce(f"attention half H={H} D={D} {lengths}")
        x, residual = server.rows(M, H)
        step = [dev(a) for a in server.step(lengths, M)]
        before = m["k_cache"].clone(), m["v_cache"].clone()
        _check(m, before, x, residual, step, window, sinks, _half(twl, m, x, residual, *step, window, sinks))

    announce(f"attention half captured H={H} D={D}")
    M = 4  # three sequences and a row of padding
    x, residual = server.rows(M, H)
    step = [dev(a) for a in server.step([1, 1, 1], M)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the linear layer keeps its workspace by stream: made before the capture
        _half(twl, m, x, residual, *step, window, sinks)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept = _half(twl, m, x, residual, *step, window, sinks)
    for lengths in ([1, 1, 1], [1, 0, 2], [1, 1, 1], [0, 4, 0]):
        for t, new in zip([x, residual] + step, server.rows(M, H) + [dev(a) for a in server.step(lengths, M)]):
            t.copy_(new)
        before = m["k_cache"].clone(), m["v_cache"].clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        after = m["k_cache"].clone(), m["v_cache"].clone()
        m["k_cache"].copy_(before[0])
        m["v_cache"].copy_(before[1])
        eager = _half(twl, m, x, residual, *step, window, sinks)
        for name in eager:
            assert torch.equal(kept[name], eager[name]), name
        assert torch.equal(after[0], m["k_cache"]) and torch.equal(after[1], m["v_cache"])
        _check(m, before, x, residual, step, window, sinks, eager)


def test_two_streams_at_once(twl):
    """Two batches of one cache on two streams, their workspaces each their own."""
    a = test_gpu_attention._case(1, [(1, 9000), (1, 5000)], 8, 2, 128, 64)
    b = dict(a, q=torch.randn_like(a["q"]))
    want = [test_gpu_attention._run(twl, c) for c in (a, b)]
    x = [torch.randint(-128, 128, (n, 5120), dtype=torch.int8, device="cuda") for n in (40, 60)]
    w = torch.randint(-128, 128, (1000, 5120), dtype=torch.int8, device="cuda")
    want_i = [twl.int8_linear(t, None, w, None, out_dtype=torch.int32) for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, got_i = [[], []], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(test_gpu_attention._run(twl, (a, b)[i]))
                got_i[i].append(twl.int8_linear(x[i], None, w, None, out_dtype=torch.int32))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])
        assert all(torch.equal(t, want_i[i]) for t in got_i[i])


@pytest.mark.parametrize("M,N,K", [(150, 2 ** 24 - 3, 32), (200, 2 ** 24, 16)])
def test_int8_outputs_past_32_bits(twl, M, N, K):
    announce(f"int8_linear {M} x {K} -> {N}")
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    out = twl.int8_linear(x, None, w, None, out_dtype=torch.int32)
    for n in (0, N // 2 - 500, N - 1000):
        assert torch.equal(out[:, n:n + 1000], (x.double() @ w[n:n + 1000].double().T).int())
    assert torch.equal(out[M - 1], (w.float() * x[M - 1].float()).sum(1).int())  # sums below 2^24: exact in fp32


def test_rope_rows_past_32_bits(twl):
    M, n_q, n_kv, D = 600_000, 14, 1, 256
    announce(f"qk_norm_rope {M} tokens")
    qkv = torch.randn(M, (n_q + 2 * n_kv) * D, dtype=torch.bfloat16, device="cuda")
    positions = torch.arange(M, dtype=torch.int32, device="cuda") % N_POS
    cos_sin, w = dev(test_gpu_rope._table(N_POS, D)), torch.ones(D, dtype=torch.bfloat16, device="cuda")
    got = twl.qk_norm_rope(qkv, positions, cos_sin, n_q, n_kv, q_weight=w, k_weight=w)
    for rows in (slice(0, 100), slice(M - 300_000, M - 299_900), slice(M - 100, M)):
        alone = twl.qk_norm_rope(qkv[rows], positions[rows].clone(), cos_sin, n_q, n_kv, q_weight=w, k_weight=w)
        assert all(torch.equal(a[rows], b) for a, b in zip(got, alone))


@pytest.mark.parametrize("D", [128, 256])
def test_attention_rows_past_32_bits(twl, D):
    T, n_q, page = 2 ** 25 // D, 64, 64
    T += 1000
    announce(f"window_attention {T} tokens of {n_q} heads of {D}")
    q = torch.randn(T, n_q, D, dtype=torch.bfloat16, device="cuda")
    pages = -(-T // page)
    k = torch.randn(pages, 1, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.randn(pages, 1, page, D, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = twl.window_attention(q, k, v, table, dev(np.array([0, T], np.int32)), dev(np.array([T], np.int32)), window=1)
    want = v.view(-1, D)[:T]  # each row sees its own key alone
    assert all(torch.equal(out[:, h], want) for h in range(n_q))
