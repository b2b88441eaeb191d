"""window_attention on the GPU against the float64 oracle, element by element.

The bound.  u = 2^-24.  A score sums D fp32 products: off by at most (D + 4) u of
S = scale sum |q k|, its product with log2 e and the difference from the maximum by 4 u S more, and
the exponential by 2^-22 relative: a weight is within e = (2 D + 16) u S + 2^-21 of its value (S the row's
largest), and, rounded to bf16, within 2^-8 + e.  out is a quotient whose weights all have such a factor
1 + d, above and below: it moves by sum w d (v - out), at most max|d| (W + |out|) with W = sum w |v| / sum w,
and in second order by 2^-6 of that.  The fp32 sums of n keys add (n + 64) u.  Then one rounding: 2^-8 |out|."""
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


def _bf(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().cuda()


def _case(seed, lengths, n_q, n_kv, D, page, spare_rows=0, spare_pages=2, wide=0, garbage=True):
    """Sequences (new tokens, context) over shuffled pages; what no sequence holds is NaN."""
    rng = np.random.default_rng(seed)
    need = [-(-kv // page) for _, kv in lengths]
    n_pages = sum(need) + spare_pages
    order = rng.permutation(n_pages)
    table = np.full((len(lengths), max(need + [1]) + wide), -1, np.int32)
    k = rng.standard_normal((n_pages, n_kv, page, D)).astype(np.float32)
    v = rng.standard_normal((n_pages, n_kv, page, D)).astype(np.float32)
    held = np.zeros((n_pages, page), bool)
    at = 0
    for b, (_, kv) in enumerate(lengths):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        j = np.arange(kv)
        held[table[b, j // page], j % page] = True
    if garbage:
        for c in (k, v):
            c.transpose(0, 2, 1, 3)[~held] = np.nan
    starts = np.concatenate([[0], np.cumsum([n for n, _ in lengths])]).astype(np.int32)
    T = int(starts[-1]) + spare_rows
    return dict(q=_bf(rng.standard_normal((T, n_q, D))), k_cache=_bf(k), v_cache=_bf(v), page_table=dev(table), q_start=dev(starts),
                kv_len=dev(np.array([kv for _, kv in lengths], np.int32)))


def _np(t):
    return host(t.float()).astype(np.float64)


def _check(c, out, scale=None, window=0, sinks=0):
    D = c["q"].shape[2]
    scale = D ** -0.5 if scale is None else scale
    k, v = np.nan_to_num(_np(c["k_cache"]), nan=0, posinf=0, neginf=0), np.nan_to_num(_np(c["v_cache"]), nan=0, posinf=0, neginf=0)
    want, mag, size = A.window_attention(_np(c["q"]), k, v, host(c["page_table"]), host(c["q_start"]), host(c["kv_len"]), scale, window, sinks)
    rows = np.isfinite(want[:, 0, 0])
    got, want, mag, size = _np(out)[rows], want[rows], mag[rows], size[rows]
    n = int(host(c["kv_len"]).max(initial=0))
    e = 2.0 ** -8 + (2 * D + 16) * U * size + 2.0 ** -21 + (n + 64) * U
    delta = e * (mag + np.abs(want)) * (1 + 2.0 ** -6)
    tol = delta + (np.abs(want) + delta) * 2.0 ** -8 + 2.0 ** -134
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (float(np.max(err / tol)), np.unravel_index(np.argmax(err / tol), err.shape))


def _run(twl, c, **kw):
    return twl.window_attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["q_start"], c["kv_len"], **kw)


DECODE = [(1, 1), (1, 2), (1, 31), (1, 32), (1, 33), (1, 100), (1, 517)]
DRAFTS = [(4, 4), (3, 70), (0, 9), (5, 300), (1, 1), (8, 8), (2, 1000)]
PROMPTS = [(130, 130), (1, 40), (0, 0), (77, 77), (200, 333), (64, 64), (65, 640)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 3), (40, 4), (64, 0), (250, 40), (100000, 2)])
@pytest.mark.parametrize("D,n_q,n_kv,page", [(64, 6, 2, 16), (128, 5, 1, 64), (256, 4, 2, 32), (128, 3, 3, 16), (64, 20, 1, 128)])
@pytest.mark.parametrize("lengths", [DECODE, DRAFTS, PROMPTS], ids=["decode", "drafts", "prompts"])
def test_values(twl, lengths, D, n_q, n_kv, page, window, sinks):
    announce(f"window_attention {lengths} {n_q}/{n_kv} x {D} pages of {page} window {window} sinks {sinks}")
    c = _case(D + window, lengths, n_q, n_kv, D, page)
    _check(c, _run(twl, c, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[(1, 9000)], [(1, 5001), (1, 40), (1, 12345)], [(6, 7000), (1, 300)], [(700, 2000)], [(1, 6000), (513, 600), (1, 33)],
                                     [(300, 300)] * 3], ids=str)
def test_long(twl, lengths, D):
    for window, sinks in ((0, 0), (1500, 5)):
        c = _case(D, lengths, 10, 2, D, 64)
        _check(c, _run(twl, c, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,kv", [(1, 3000), (3, 500), (40, 400), (300, 300), (200, 900)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 1), (33, 0), (100, 17), (129, 70)])
def test_which_keys_are_seen(twl, D, n, kv, window, sinks):
    """Equal scores and values that count: every output is (keys seen with j % D == d) /
    (keys seen), weights and their sums exact, one quotient and one rounding."""
    c = _case(1, [(n, kv), (1, 50)], 3, 1, D, 16)
    c["q"].zero_()
    v = np.full(c["v_cache"].shape, np.nan, np.float32)
    table = host(c["page_table"])
    for b, m in enumerate((kv, 50)):
        for j in range(m):
            v[table[b, j // 16], 0, j % 16] = np.arange(D) == j % D
    c["v_cache"] = _bf(v)
    got = _np(_run(twl, c, window=window, sinks=sinks))[:n]
    seen = A.mask(n, kv, window, sinks)
    count = np.stack([seen[:, d::D].sum(1) if d < kv else np.zeros(n) for d in range(D)], 1)
    want = (count / seen.sum(1, keepdims=True))[:, None, :]
    assert (np.abs(got - want) <= want * (2.0 ** -8 + 2.0 ** -20)).all()


@pytest.mark.parametrize("page", [16, 32, 256, 1024])
def test_page_sizes(twl, page):
    c = _case(2, [(1, 1500), (30, 90), (150, 700)], 4, 2, 64, page)
    _check(c, _run(twl, c, window=300, sinks=20), window=300, sinks=20)


@pytest.mark.parametrize("n", [1, 5, 150])
def test_rows_without_keys_and_lengths_of_zero(twl, n):
    """More new tokens than context: positions below zero see nothing, their rows are 0."""
    c = _case(3, [(n, n), (n, max(1, n // 2)), (n, 0), (0, 5), (0, 0)], 4, 2, 128, 16)
    c["kv_len"] = dev(np.array([n, n // 2, -3, 5, 0], np.int32))
    out = _run(twl, c)
    _check(c, out)
    assert (out[2 * n:] == 0).all() and (out[n:n + n - n // 2] == 0).all()


@pytest.mark.parametrize("n", [1, 4, 200])
def test_pages_that_are_none(twl, n):
    """Freed pages (-1), numbers outside the cache and a context longer than the table."""
    c = _case(4, [(n, 700), (n, 300), (n, 260)], 6, 2, 64, 16, garbage=False)  # kv_len grows below: every slot of a page counts
    table = host(c["page_table"]).copy()
    table[0, 1:20] = -1
    table[1, 3], table[1, 5], table[1, -25] = c["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31
    c["page_table"] = dev(table)
    c["kv_len"] = dev(np.array([700, 300, 16 * table.shape[1] + 40], np.int32))
    for window, sinks in ((0, 0), (300, 8)):
        _check(c, _run(twl, c, window=window, sinks=sinks), window=window, sinks=sinks)
    table[:] = -1
    c["page_table"] = dev(table)
    assert (_run(twl, c) == 0).all()


@pytest.mark.parametrize("n", [1, 3, 140])
def test_freed_pages_behind_the_window_are_not_read(twl, n):
    c = _case(5, [(n, 900), (n, 500)], 4, 1, 128, 16)
    window, sinks = 200, 4
    want = _run(twl, c, window=window, sinks=sinks)
    table = host(c["page_table"]).copy()
    for b, kv in enumerate((900, 500)):
        first = (kv - n - window + 1) // 16
        if first > 1:
            table[b, 1:first] = -1
    c["page_table"] = dev(table)
    assert torch.equal(_run(twl, c, window=window, sinks=sinks), want)


@pytest.mark.parametrize("lengths", [[(1, 70)] * 3, [(90, 90), (1, 20)], []], ids=str)
def test_rows_behind_the_last_sequence_stay(twl, lengths):
    c = _case(6, lengths, 4, 2, 64, 16, spare_rows=40)
    out = torch.full_like(c["q"], 5.0)
    assert _run(twl, c, out=out) is out
    used = sum(n for n, _ in lengths)
    assert (out[used:] == 5).all()
    _check(c, out)


def test_starts_outside_the_rows(twl):
    c = _case(7, [(3, 30), (60, 60), (2, 9)], 4, 2, 64, 16)
    c["q_start"] = dev(np.array([0, 3, 63, 2 ** 31 - 1], np.int32))
    _check(c, _run(twl, c))
    c["q_start"] = dev(np.array([-5, 3, 63, 65], np.int32))
    _check(c, _run(twl, c))


@pytest.mark.parametrize("lengths", [[(1, 300)] * 4, [(1, 4000)], [(260, 260)]], ids=str)
def test_other_scales_and_large_scores(twl, lengths):
    for scale in (0.5, -0.2, 0.0):
        c = _case(8, lengths, 4, 2, 64, 16)
        _check(c, _run(twl, c, scale=scale), scale=scale)
    c = _case(9, lengths, 4, 2, 128, 16)
    c["q"] *= 30.0  # one key takes nearly all
    _check(c, _run(twl, c))
    c["q"].fill_(-100.0)
    c["k_cache"] = torch.where(c["k_cache"].isnan(), c["k_cache"], 100.0 + 0 * c["k_cache"])  # all scores near -1e6
    _check(c, _run(twl, c))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[(1, 300)] * 4, [(1, 4000)], [(260, 260)], [(200, 3000)]], ids=str)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_near_the_largest(twl, lengths, D, sign):
    """Scores of about 2^113 with room for fp32's sums: equal ones weigh alike, and of two sizes the larger takes all."""
    c = _case(17, lengths, 4, 2, D, 16)
    k_nan = c["k_cache"].isnan()
    c["q"].fill_(2.0 ** 55)
    c["k_cache"] = torch.where(k_nan, c["k_cache"], torch.full_like(c["k_cache"], sign * 2.0 ** 55))
    got = _run(twl, c)
    equal = _run(twl, dict(c, q=torch.zeros_like(c["q"])))  # all scores 0
    assert torch.equal(got, equal)
    _check(dict(c, q=torch.zeros_like(c["q"])), got)
    top = torch.where(torch.arange(16, device="cuda")[None, None, :, None] == 0, c["k_cache"] * (1.0 + 0.25 * sign), c["k_cache"])
    got = _run(twl, dict(c, k_cache=top))  # each page's first key wins
    zero_one = torch.where(k_nan, c["k_cache"], torch.where(torch.arange(16, device="cuda")[None, None, :, None] == 0, 6.0, 0.0).bfloat16())
    _check(dict(c, q=torch.full_like(c["q"], 6.0), k_cache=zero_one), got)


@pytest.mark.parametrize("n", [1, 3, 150])
def test_lengths_beyond_the_table(twl, n):
    """What the table does not hold is not seen, at positions up to 2^30 (longer lengths count as that)."""
    c = _case(18, [(n, 512), (1, 100)], 4, 2, 64, 16)
    c["kv_len"] = dev(np.array([512 + n, 100], np.int32))  # every new token behind the table
    want = _run(twl, c)
    _check(c, want)
    for kv in (100000, 2 ** 30, 2 ** 30 + 5, 2 ** 31 - 1):
        c["kv_len"] = dev(np.array([kv, 100], np.int32))
        assert torch.equal(_run(twl, c), want)
    got = _run(twl, c, window=2 ** 30, sinks=7)
    assert torch.equal(got[n:], want[n:])
    sinks = _run(twl, c, window=50, sinks=7)
    c["kv_len"] = dev(np.array([512 + n + 50, 100], np.int32))
    want = _run(twl, c, window=50, sinks=7)
    _check(c, want, window=50, sinks=7)
    assert torch.equal(sinks, want)
    assert (_run(twl, c, window=1)[:n] == 0).all()


@pytest.mark.parametrize("n_q,n_kv", [(4, 2), (40, 1)])
def test_starts_that_decrease_stay_in_bounds(twl, n_q, n_kv):
    c = _case(19, [(3, 30), (60, 60), (2, 9), (100, 200), (1, 5)], n_q, n_kv, 64, 16, spare_rows=20)
    T = c["q"].shape[0]
    guard = torch.full((T + 64, n_q, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for starts in ([0, 100, 5, 80, 2, 166], [166, 0, 166, 0, 166, 0], [50, 40, 30, 20, 10, 0], [0, 0, 2 ** 31 - 1, -2 ** 31, 63, 64]):
        c["q_start"] = dev(np.array(starts, np.int32))
        _run(twl, c, out=guard[32:32 + T])
        assert (guard[:32] == 7).all() and (guard[32 + T:] == 7).all()


def test_most_sequences(twl):
    c = _case(20, [(1, 40), (2, 2100), (1, 7)], 2, 1, 64, 16)
    want = _run(twl, c)
    _check(c, want)
    for B in (4096, 65536):
        starts, lens = np.zeros(B + 1, np.int32), np.zeros(B, np.int32)
        table = np.full((B, c["page_table"].shape[1]), -1, np.int32)
        at = [5, B // 2, B - 3]
        for i, (b, n) in enumerate(zip(at, (1, 2, 1))):
            starts[b + 1:] += n
            lens[b], table[b] = int(c["kv_len"][i]), host(c["page_table"])[i]
        many = dict(c, q_start=dev(starts), kv_len=dev(lens), page_table=dev(table))
        _check(c, _run(twl, many))  # the same rows and keys


@pytest.mark.parametrize("n", [1, 200])
def test_values_not_finite_of_one_sequence_stay_there(twl, n):
    c = _case(10, [(n, 300), (n, 400)], 4, 2, 128, 16)
    want = _run(twl, c)
    page = int(c["page_table"][0, 2])
    c["v_cache"][page, 0, 3] = float("inf")
    c["k_cache"][page, 1, 3] = float("nan")
    got = _run(twl, c)
    assert torch.equal(got[n:], want[n:])
    assert not torch.isfinite(got[n - 1]).all()


@pytest.mark.parametrize("lengths", [[(1, 100), (1, 7)], [(1, 9000)], [(100, 300), (1, 50)]], ids=str)
def test_stream_workspace_and_repeats(twl, lengths):
    c = _case(11, lengths, 10, 2, 128, 64)
    T, B = c["q"].shape[0], len(lengths)
    need = twl.attention_workspace_bytes(T, B, 10, 2, 128, 64, c["page_table"].shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = _run(twl, c, workspace=ws, stream=side)
    b = _run(twl, c, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(c, a)
    assert torch.equal(a, b)
    if need:
        with pytest.raises(twl.TwlError, match="workspace"):
            _run(twl, c, workspace=ws[:need - 16])


@pytest.mark.parametrize("window", [0, 200])
def test_graph_serves_other_lengths(twl, window):
    c = _case(12, [(1, 3000), (3, 40), (80, 500), (1, 64)], 10, 2, 64, 16, garbage=False)
    _run(twl, c, window=window)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(twl, c, window=window, sinks=4)
    for starts, kv in [([0, 1, 4, 84, 85], [2999, 39, 499, 63]), ([0, 0, 40, 45, 85], [7, 500, 5, 64]), ([0, 85, 85, 85, 85], [2000, 0, 0, 0]),
                       ([0, 1, 2, 3, 4], [2500, 1, 450, 33])]:
        c["q_start"].copy_(torch.tensor(starts, dtype=torch.int32))
        c["kv_len"].copy_(torch.tensor(kv, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.zeros_like(out)
        _run(twl, c, window=window, sinks=4, out=eager)
        assert torch.equal(out, eager)
        _check(c, out, window=window, sinks=4)


def test_many_sequences(twl):
    rng = np.random.default_rng(0)
    for most in (1, 40):
        lengths = [(int(n), int(n) + int(k)) for n, k in zip(rng.integers(0, most + 1, 150), rng.integers(0, 60, 150))]
        c = _case(13, lengths, 2, 1, 64, 16)
        _check(c, _run(twl, c, window=30, sinks=2), window=30, sinks=2)


def test_cache_past_32_bit_offsets(twl):
    pages = 2 ** 31 // (8 * 64 * 128) + 5
    c = _case(14, [(1, 150), (70, 130)], 8, 8, 128, 64, garbage=False)
    small_k, small_v, table = c["k_cache"], c["v_cache"], host(c["page_table"]).copy()
    want = _run(twl, c)
    c["k_cache"] = torch.zeros((pages, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
    c["v_cache"] = torch.zeros((pages, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
    far = np.where(table >= 0, pages - 1 - table, -1).astype(np.int32)
    for t in table[table >= 0]:
        c["k_cache"][pages - 1 - int(t)], c["v_cache"][pages - 1 - int(t)] = small_k[int(t)], small_v[int(t)]
    c["page_table"] = dev(far)
    assert torch.equal(_run(twl, c), want)


def test_empty_and_refusals(twl):
    c = _case(15, [(2, 20)], 4, 2, 64, 16)
    none = _run(twl, dict(c, q=c["q"][:0]))
    assert none.shape == (0, 4, 64)
    call = lambda **kw: _run(twl, dict(c, **{k: kw.pop(k) for k in list(kw) if k in c}), **kw)  # noqa: E731
    for kw, error, word in [
            (dict(q=c["q"][0]), ValueError, "q must be"), (dict(k_cache=c["k_cache"][0]), ValueError, "k_cache"),
            (dict(v_cache=c["v_cache"][:1]), ValueError, "v_cache"), (dict(q=c["q"].float()), TypeError, "q has dtype"),
            (dict(kv_len=c["kv_len"].long()), TypeError, "kv_len"), (dict(q_start=c["q_start"][:1]), ValueError, "q_start"),
            (dict(page_table=c["page_table"][0]), ValueError, "page_table"), (dict(q=c["q"][:, :3].contiguous()), twl.TwlError, "multiple"),
            (dict(window=-1), twl.TwlError, "window"), (dict(sinks=-1), twl.TwlError, "sinks"), (dict(scale=float("nan")), twl.TwlError, "scale"),
            (dict(q=c["q"].clone().requires_grad_()), ValueError, "requires grad"), (dict(out=c["q"]), twl.TwlError, "overlaps"),
            (dict(k_cache=c["k_cache"][:, :, :8].contiguous(), v_cache=c["v_cache"][:, :, :8].contiguous()), twl.TwlError, "page size"),
            (dict(q=c["q"][:, :, :32].contiguous(), k_cache=c["k_cache"][..., :32].contiguous(), v_cache=c["v_cache"][..., :32].contiguous()),
             twl.TwlError, "head size")]:
        with pytest.raises(error, match=word):
            call(**kw)
    nothing = dict(c, k_cache=c["k_cache"][:0], v_cache=c["v_cache"][:0])
    assert (_run(twl, nothing) == 0).all()
