"""int8_linear's kernels one by one: every tile and every number of splits of K that a size can
get, with more stages of K than a tile keeps in flight, a K that ends inside a stage, rows and
columns that end inside a tile and rows of the output of each alignment.

tests/test_attention_plans_host.py holds that each size gets the kernel named here.  Sums against
float64 products on the device (below 2^53: exact); the bound of scaled outputs is that of
test_gpu_int8.py."""
import pytest

from tests.gpu_helpers import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TILES = ["256x256", "192x256", "256x128", "128x128", "64x128", "64x64"]

# tile, splits: sizes M, N, K with N a multiple of 8, of 4 and odd
TILED = {
    (0, 1): [(202, 36840, 560), (468, 30668, 1040), (2815, 9219, 2064)],
    (0, 2): [(194, 17480, 11360), (193, 16452, 11280), (194, 16575, 11040)],
    (0, 4): [(6687, 272, 11408), (198, 8572, 11424), (193, 8195, 12448)],
    (0, 8): [(6370, 144, 26784), (6370, 148, 26784), (6370, 145, 26784)],
    (1, 1): [(143, 33744, 560), (130, 33284, 624), (134, 52763, 1040), (4096, 17408, 5120)],
    (1, 2): [(136, 22408, 6336), (140, 22468, 7616), (132, 23255, 6112)],
    (1, 4): [(130, 8856, 10128), (138, 8452, 10112), (132, 8313, 10336)],
    (1, 8): [(5672, 136, 11072), (5702, 132, 12224), (133, 5485, 9808)],
    (2, 1): [(131, 21896, 560), (225, 24620, 1040), (138, 23235, 528)],
    (2, 2): [(8384, 272, 13488), (8384, 276, 13488), (8384, 273, 13488)],
    (2, 4): [(3283, 272, 10176), (5560, 132, 10560), (5471, 129, 8624)],
    (2, 8): [(4140, 68, 14944), (4219, 65, 15296)],
    (3, 1): [(65, 17528, 560), (257, 9316, 2064), (69, 17554, 528)],
    (3, 2): [(68, 9016, 3216), (70, 8316, 3408), (68, 8217, 3648)],
    (3, 4): [(4427, 72, 6064), (4161, 68, 6128), (65, 4226, 6048)],
    (3, 8): [(66, 2176, 5344), (2230, 68, 5024), (2053, 69, 5024)],
    (4, 1): [(65, 8992, 528), (66, 8580, 592), (65, 8245, 544)],
    (4, 2): [(35, 16680, 7872), (36, 17948, 7824), (34, 16479, 7760)],
    (4, 4): [(37, 9336, 10416), (35, 8276, 10176), (35, 8198, 9760)],
    (4, 8): [(41, 4224, 9936), (34, 4724, 8736), (35, 4129, 8048)],
    (5, 1): [(37, 32, 656), (36, 36, 704), (333, 4001, 2064)],
    (5, 2): [(4166, 32, 3824), (2216, 68, 3520), (4249, 34, 3504)],
    (5, 4): [(34, 32, 3360), (35, 36, 3056), (34, 34, 3056)],
    (5, 8): [(37, 32, 6032), (35, 36, 7216), (36, 33, 6256)],
}
# tiles of 16 channels and of 16 tokens of a workgroup
ROWS = {
    (1, 1): [(3, 4001, 2064), (16, 333, 1040)],
    (1, 2): [(17, 1000, 528), (32, 4095, 4112)],
    (2, 1): [(5, 4101, 1104), (16, 5000, 2096)],
    (2, 2): [(17, 4097, 1040), (31, 32767, 560)],
    (4, 2): [(24, 32771, 1040), (32, 40008, 528), (17, 65536, 2064)],
}


@pytest.fixture(scope="module")
def twl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_weight_linear_block_amd as m
    m.library()
    return m


def _check(twl, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x, w = (torch.randint(-128, 128, (n, K), dtype=torch.int8, device="cuda", generator=g) for n in (M, N))
    acc = x.double() @ w.double().T
    got = torch.full((M + 2, N), 7, dtype=torch.int32, device="cuda")
    out = got.view(-1)[:M * N].view(M, N)
    twl.int8_linear(x, None, w, None, out=out)
    assert torch.equal(out, acc.int())
    assert (got.view(-1)[M * N:] == 7).all()
    a, s = (torch.rand(n, device="cuda", generator=g) + 0.01 for n in (M, N))
    bias = torch.randn(N, device="cuda", generator=g) * 100
    y = acc * a.double()[:, None] * s.double()
    for b in (None, bias):
        want = y if b is None else y + b.double()
        for dtype in (torch.float32, torch.bfloat16):
            tol = 4 * U * y.abs() + U * want.abs()
            if dtype == torch.bfloat16:
                tol += (want.abs() + tol) * 2.0 ** -8
            got = twl.int8_linear(x, a, w, s, bias=b, out_dtype=dtype)
            assert ((got.double() - want).abs() <= tol).all(), dtype


@pytest.mark.parametrize("tile,splits", TILED, ids=lambda v: str(v))
def test_tiles(twl, tile, splits):
    for M, N, K in TILED[tile, splits]:
        announce(f"int8_linear {M} x {K} -> {N}: tile {TILES[tile]}, {splits} splits")
        _check(twl, M, N, K)


@pytest.mark.parametrize("rt,mt", ROWS)
def test_rows(twl, rt, mt):
    for M, N, K in ROWS[rt, mt]:
        announce(f"int8_linear {M} x {K} -> {N}: {16 * rt} channels and {16 * mt} tokens a workgroup")
        _check(twl, M, N, K)
