"""window_attention's kernel for many rows at the masks, lengths and pages where it can go wrong,
alone and beside short sequences, with its keys split and not.

Which kernel a call takes goes by estimated time: rows behind the last sequence and entries behind
a table's last page, which cost the oracle nothing, make calls of few rows and keys take
this one.  tests/test_attention_plans_host.py holds what each call here takes.  Oracle and
bound are those of test_gpu_attention.py."""
import numpy as np
import pytest

import oracle.attention_oracle as A
from tests import test_gpu_attention as S
from tests.gpu_helpers import announce, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# (D, n_q, n_kv, page): groups that divide a tile's 128 rows and such that do not
SHAPES = [(64, 6, 2, 16), (64, 20, 1, 128), (128, 5, 1, 64), (128, 3, 3, 16), (256, 4, 2, 32), (256, 7, 1, 16)]
ONE = {64: (64, 4, 2, 16), 128: (128, 5, 1, 16), 256: (256, 3, 1, 16)}
ALONE = [[(130, 130)], [(77, 333)], [(200, 1000)], [(1, 70)], [(3, 500)], [(150, 60)]]
BESIDE = [[(130, 130), (1, 40), (0, 0), (77, 77), (200, 333), (64, 64), (65, 640)], [(1, 900), (300, 1200), (5, 300), (90, 40), (0, 7)]]
WINDOWS = [(0, 0), (1, 0), (7, 3), (40, 4), (64, 64), (20, 70), (250, 40), (100, 200), (100000, 2)]
LONG = [[(200, 3000)], [(130, 2200), (1, 3000), (300, 900)]]
LONG_WINDOWS = [(0, 0), (1500, 5), (2000, 130)]


def form(D, split):
    """(rows x query heads, keys of the table) that make a call take the kernel for many rows: with more tiles than
    half the device's places, with few enough tiles and enough keys for two splits, or (2) for several."""
    if split == 2:
        return {64: 7000, 128: 5000, 256: 3000}[D], 16384
    return ({64: 32000, 128: 24000, 256: 12000} if split else {64: 60000, 128: 36000, 256: 18000})[D], 4096 if split else 0


def case(seed, lengths, shape, split, **kw):
    D, n_q, n_kv, page = shape
    rows, keys = form(D, split)
    used, widest = sum(n for n, _ in lengths), max(-(-kv // page) for _, kv in lengths)
    return S._case(seed, lengths, n_q, n_kv, D, page, spare_rows=max(0, -(-rows // n_q) - used), wide=max(0, keys // page - max(widest, 1)), **kw)


def calls():
    """What the tests below run (and, with splits, a few windows whose plan has none): (lengths, shape, split, window, sinks, whether the plan has splits)."""
    for shape in SHAPES:
        for lengths in ALONE + BESIDE:
            for window, sinks in WINDOWS:
                yield lengths, shape, False, window, sinks, False
        for lengths in LONG:
            for window, sinks in LONG_WINDOWS:
                yield lengths, shape, True, window, sinks, True
            yield lengths, shape, 2, 0, 0, True
    for shape in GROUPS:
        for window, sinks in ((0, 0), (33, 5)):
            yield GROUPED, shape, False, window, sinks, False
    for shape in ONE.values():
        for lengths in ([(n, kv)] for n, kv in SEEN):
            for window, sinks in SEEN_WINDOWS:
                yield lengths, shape, False, window, sinks, False
            yield lengths, shape, True, 0, 0, True
        for split in (False, True):
            for lengths in (EMPTY, FREED, FINITE, EQUAL, BEYOND, SERVED, [(3, 30), (60, 60), (2, 9), (100, 200), (1, 5)]):
                yield lengths, shape, split, 0, 0, split
                for window, sinks in () if split else ((20, 3), (50, 7), (100, 4), (300, 8)):
                    yield lengths, shape, split, window, sinks, False
        yield EXTREME, shape, False, 0, 0, False
        yield EXTREME, shape, True, 0, 0, True
        for page in PAGES:
            for window, sinks in ((0, 0), (300, 20)):
                yield PAGED, (*shape[:3], page), False, window, sinks, False


@pytest.fixture(scope="module")
def twl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_weight_linear_block_amd as m
    m.library()
    return m


def run(twl, c, **kw):
    """The call, into an `out` whose rows behind the last sequence have to stay as they were."""
    out = torch.full_like(c["q"], 5.0)
    S._run(twl, c, out=out, **kw)
    used = int(c["q_start"].max().clamp(0, c["q"].shape[0]))
    assert (out[used:] == 5).all()
    return out[:used]


def check(c, out, **kw):
    S._check(dict(c, q=c["q"][:out.shape[0]]), out, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("lengths", ALONE + BESIDE, ids=str)
def test_values(twl, lengths, shape):
    c = case(sum(shape), lengths, shape, False)
    for window, sinks in WINDOWS:
        announce(f"window_attention, many rows: {lengths} {shape} window {window} sinks {sinks}")
        check(c, run(twl, c, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("lengths", LONG, ids=str)
def test_splits(twl, lengths, shape):
    c = case(sum(shape) + 1, lengths, shape, True)
    for window, sinks in LONG_WINDOWS:
        announce(f"window_attention, many rows, split: {lengths} {shape} window {window} sinks {sinks}")
        check(c, run(twl, c, window=window, sinks=sinks), window=window, sinks=sinks)
    c = case(sum(shape) + 2, lengths, shape, 2)
    announce(f"window_attention, many rows, more splits: {lengths} {shape}")
    check(c, run(twl, c))


SEEN = [(1, 3000), (3, 500), (40, 400), (300, 300), (200, 900)]
SEEN_WINDOWS = [(0, 0), (1, 1), (33, 0), (64, 64), (63, 65), (10, 200), (100, 17), (129, 70), (300, 1)]


@pytest.mark.parametrize("D", sorted(ONE))
@pytest.mark.parametrize("n,kv", SEEN)
def test_which_keys_are_seen(twl, n, kv, D):
    """Equal scores and values that count, as in test_gpu_attention.py: every weight and sum is exact."""
    for split in (False, True):
        c = case(1, [(n, kv)], ONE[D], split)
        c["q"].zero_()
        v = np.full(c["v_cache"].shape, np.nan, np.float32)
        page, j = ONE[D][3], np.arange(kv)
        v[host(c["page_table"])[0, j // page], :, j % page] = (np.arange(D) == j[:, None] % D)[:, None, :]
        c["v_cache"] = S._bf(v)
        for window, sinks in [(0, 0)] if split else SEEN_WINDOWS:
            got = S._np(run(twl, c, window=window, sinks=sinks))
            seen = A.mask(n, kv, window, sinks)
            count = np.stack([seen[:, d::D].sum(1) if d < kv else np.zeros(n) for d in range(D)], 1)
            want = (count / seen.sum(1, keepdims=True))[:, None, :]
            assert (np.abs(got - want) <= want * (2.0 ** -8 + 2.0 ** -20)).all(), (split, window, sinks)


EMPTY = [(150, 150), (150, 70), (150, 1), (0, 5), (0, 1)]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D", sorted(ONE))
def test_rows_without_keys_and_lengths_of_zero(twl, D, split):
    c = case(3, EMPTY, ONE[D], split)
    c["kv_len"] = dev(np.array([150, 70, -3, 5, 0], np.int32))
    for window, sinks in ((0, 0), (30, 3)):
        out = run(twl, c, window=window, sinks=sinks)
        check(c, out, window=window, sinks=sinks)
        assert (out[300:] == 0).all() and (out[150:230] == 0).all()
    table = torch.full_like(c["page_table"], -1)
    assert (run(twl, dict(c, page_table=table)) == 0).all()
    nothing = dict(c, k_cache=c["k_cache"][:0], v_cache=c["v_cache"][:0])
    assert (run(twl, nothing) == 0).all()


FREED = [(200, 700), (140, 300), (90, 260), (2, 500)]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D", sorted(ONE))
def test_pages_that_are_none(twl, D, split):
    """Freed pages, numbers outside the cache, and freed ones behind the window, whose keys are not read."""
    c = case(4, FREED, ONE[D], split, garbage=False)
    table = host(c["page_table"]).copy()
    table[0, 1:20] = -1
    table[1, 3], table[1, 5], table[1, 15], table[2, 0] = c["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31, -1
    table[3, 2:9] = -7
    bad = dict(c, page_table=dev(table))
    for window, sinks in ((0, 0), (300, 8), (64, 100)):
        check(bad, run(twl, bad, window=window, sinks=sinks), window=window, sinks=sinks)
    window, sinks = 100, 4
    want = run(twl, c, window=window, sinks=sinks)
    check(c, want, window=window, sinks=sinks)
    table = host(c["page_table"]).copy()
    for b, (n, kv) in enumerate(FREED):
        table[b, 1:max(1, (kv - n - window + 1) // 16)] = -1
    assert torch.equal(run(twl, dict(c, page_table=dev(table)), window=window, sinks=sinks), want)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D", sorted(ONE))
def test_scales_and_large_scores(twl, D, split):
    c = case(8, FREED, ONE[D], split)
    for scale in (0.5, -0.2, 0.0, 2.0, -3.0):
        check(c, run(twl, c, scale=scale), scale=scale)
    large = dict(c, q=c["q"] * 30.0)  # one key takes nearly all
    check(large, run(twl, large))
    same = dict(c, q=torch.full_like(c["q"], -100.0), k_cache=torch.where(c["k_cache"].isnan(), c["k_cache"], torch.full_like(c["k_cache"], 100.0)))
    check(same, run(twl, same))  # all scores near -1e6
    check(same, run(twl, same, scale=-0.5), scale=-0.5)


EQUAL = [(160, 160), (140, 900), (1, 50)]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("D", sorted(ONE))
def test_scores_near_the_largest(twl, D, sign, split):
    """Scores of about 2^113: equal ones weigh alike, and of two sizes the larger takes all."""
    c = case(17, EQUAL, ONE[D], split)
    k_nan = c["k_cache"].isnan()
    zero = dict(c, q=torch.zeros_like(c["q"]))
    equal = run(twl, zero)
    check(zero, equal)
    c["q"].fill_(2.0 ** 55)
    c["k_cache"] = torch.where(k_nan, c["k_cache"], torch.full_like(c["k_cache"], sign * 2.0 ** 55))
    assert torch.equal(run(twl, c), equal)
    first = torch.arange(16, device="cuda")[None, None, :, None] == 0
    got = run(twl, dict(c, k_cache=torch.where(first, c["k_cache"] * (1.0 + 0.25 * sign), c["k_cache"])))  # each page's first key wins
    zero_one = torch.where(k_nan, c["k_cache"], torch.where(first, 6.0, 0.0).bfloat16())
    check(dict(c, q=torch.full_like(c["q"], 6.0), k_cache=zero_one), got)


BEYOND = [(150, 512), (90, 100)]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D", sorted(ONE))
def test_lengths_beyond_the_table(twl, D, split):
    """What the table does not hold is not seen, at positions up to 2^30 (longer lengths count as that)."""
    c = case(18, BEYOND, ONE[D], split)
    keys = c["page_table"].shape[1] * 16
    c["kv_len"] = dev(np.array([keys + 150, 100], np.int32))  # every new token behind the table
    want = run(twl, c)
    check(c, want)
    for kv in (100000, 2 ** 30, 2 ** 30 + 5, 2 ** 31 - 1):
        c["kv_len"] = dev(np.array([kv, 100], np.int32))
        assert torch.equal(run(twl, c), want)
    assert torch.equal(run(twl, c, window=2 ** 30, sinks=7)[150:], want[150:])
    sinks = run(twl, c, window=50, sinks=7)
    c["kv_len"] = dev(np.array([keys + 200, 100], np.int32))
    want = run(twl, c, window=50, sinks=7)
    check(c, want, window=50, sinks=7)
    assert torch.equal(sinks, want)
    assert (run(twl, c, window=1)[:150] == 0).all()


@pytest.mark.parametrize("D", sorted(ONE))
def test_starts_that_decrease_stay_in_bounds(twl, D):
    c = case(19, [(3, 30), (60, 60), (2, 9), (100, 200), (1, 5)], ONE[D], False)
    T, n_q = c["q"].shape[:2]
    guard = torch.full((T + 64, n_q, D), 7.0, dtype=torch.bfloat16, device="cuda")
    for starts in ([0, 1000, 5, 800, 2, T], [T, 0, T, 0, T, 0], [500, 400, 300, 200, 100, 0], [0, 0, 2 ** 31 - 1, -2 ** 31, 630, 640]):
        c["q_start"] = dev(np.array(starts, np.int32))
        S._run(twl, c, out=guard[32:32 + T])
        assert (guard[:32] == 7).all() and (guard[32 + T:] == 7).all()


FINITE = [(200, 300), (150, 400), (1, 90)]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D", sorted(ONE))
def test_values_not_finite_of_one_sequence_stay_there(twl, D, split):
    c = case(10, FINITE, ONE[D], split)
    want = run(twl, c)
    check(c, want)
    page = int(c["page_table"][0, 2])
    c["v_cache"][page, 0, 3] = float("inf")
    c["k_cache"][page, 0, 4] = float("nan")
    got = run(twl, c)
    assert torch.equal(got[200:], want[200:]) and not torch.isfinite(got[199, 0]).all()
    # a key and its value that a row does not see: outside the window of all rows they change nothing
    c = case(10, FINITE, ONE[D], split)
    want = run(twl, c, window=20, sinks=3)
    table = c["page_table"]
    for b, kv, n in ((0, 300, 200), (1, 400, 150)):
        for j in (5, 47, kv - n - 20):
            c["k_cache"][int(table[b, j // 16]), :, j % 16] = float("nan")
            c["v_cache"][int(table[b, j // 16]), :, j % 16] = float("-inf")
    assert torch.equal(run(twl, c, window=20, sinks=3), want)


SERVED = [(85, 400)] * 2


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D", sorted(ONE))
def test_graph_serves_other_lengths(twl, D, split):
    c = case(12, SERVED, ONE[D], split, garbage=False)
    kw = dict(window=0 if split else 120, sinks=0 if split else 4)
    S._run(twl, c, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = S._run(twl, c, **kw)
    for starts, kv in [([0, 85, 170], [400, 400]), ([0, 1, 170], [300, 380]), ([0, 170, 170], [399, 3]), ([0, 0, 90], [9, 90]), ([0, 160, 165], [100, 400])]:
        c["q_start"].copy_(torch.tensor(starts, dtype=torch.int32))
        c["kv_len"].copy_(torch.tensor(kv, dtype=torch.int32))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = run(twl, c, **kw)
        assert torch.equal(out[:starts[-1]], eager) and (out[starts[-1]:] == 5).all()
        check(c, eager, **kw)


PAGES = [16, 32, 256, 1024]
PAGED = [(1, 1500), (130, 190), (150, 700)]


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("D", sorted(ONE))
def test_page_sizes(twl, D, page):
    shape = (*ONE[D][:3], page)
    c = case(2, PAGED, shape, False)
    for window, sinks in ((0, 0), (300, 20)):
        check(c, run(twl, c, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("D", sorted(ONE))
def test_side_stream_garbage_workspace_and_repeats(twl, D):
    shape = ONE[D]
    c = case(11, LONG[1], shape, True)
    T, B, (_, n_q, n_kv, page) = c["q"].shape[0], len(LONG[1]), shape
    need = twl.attention_workspace_bytes(T, B, n_q, n_kv, D, page, c["page_table"].shape[1])
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = run(twl, c, workspace=ws)
    b = run(twl, c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    check(c, a)
    assert torch.equal(a, b)


# groups of more query heads than a tile has rows, up to the most
GROUPS = [(64, 1024, 1, 16), (64, 300, 2, 32), (128, 257, 1, 64), (256, 129, 1, 16), (256, 512, 1, 16)]
GROUPED = [(9, 70), (2, 130), (0, 3), (1, 40)]


@pytest.mark.parametrize("shape", GROUPS, ids=str)
def test_wide_groups(twl, shape):
    announce(f"window_attention, many rows: {GROUPED} {shape}")
    shape = (shape[0], shape[1] // shape[2] * shape[2], *shape[2:])
    c = case(21, GROUPED, shape, False)
    for window, sinks in ((0, 0), (33, 5)):
        check(c, run(twl, c, window=window, sinks=sinks), window=window, sinks=sinks)


EXTREME = [(140, 300), (1, 200), (90, 90)]


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D", sorted(ONE))
def test_extreme_scales(twl, D, split, few):
    """Scales that leave all scores alike, and such that the largest one takes all.  Queries and keys of -1, 0 and 1 have
    exact scores: the output is the mean of the largest ones' values, its sum of n terms off by n 2^-24, rounded once."""
    c = S._case(22, EXTREME, *ONE[D][1:3], D, ONE[D][3]) if few else case(22, EXTREME, ONE[D], split)
    for scale in (1e-30, -1e-38, 1e-44):
        check(c, run(twl, c, scale=scale), scale=scale)
    sign = dict(c, q=c["q"].sign(), k_cache=c["k_cache"].sign())
    q, k, v = S._np(sign["q"]), np.nan_to_num(S._np(sign["k_cache"])), np.nan_to_num(S._np(c["v_cache"]))
    starts, lens, table = host(c["q_start"]), host(c["kv_len"]), host(c["page_table"])
    for scale in (1e30, -1e30, 1e34):
        out = S._np(run(twl, sign, scale=scale))
        for b in range(len(lens)):
            n, kv = starts[b + 1] - starts[b], lens[b]
            keys, values = A.gather(k, table[b], kv)[0], A.gather(v, table[b], kv)[0]
            for h in range(q.shape[1]):
                g = h // (q.shape[1] // keys.shape[0])
                score = np.where(A.mask(n, kv, 0, 0), np.sign(scale) * q[starts[b]:starts[b + 1], h] @ keys[g].T, -np.inf)
                best = score == score.max(1, keepdims=True)
                want, mag = (best @ x / best.sum(1, keepdims=True) for x in (values[g], np.abs(values[g])))
                assert (np.abs(out[starts[b]:starts[b + 1], h] - want) <= mag * (kv + 64) * S.U + np.abs(want) * 2.0 ** -7).all(), (scale, b, h)
