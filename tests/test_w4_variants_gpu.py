"""GPU tests of 4-bit products that the rule sends to kernels which the sizes in
test_w4_gpu.py do not reach, and of groups far longer than their average;
test_w4_variants_cpu.py asserts that all kernels are reached.  Whole numbers,
which have to be exact (see there)."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import test_w4_gpu as w4  # noqa: E402
from test_w4_gpu import F16, Weights, lib, rng, stacked  # noqa: E402,F401

GROUPS = [32, 64, 128, 96]

# (rows, matrices or 0 for the plain product, N, K): two row tiles with a second
# that is whole, cut and of one row; 64 columns for one and 16 rows; 32 columns and
# groups; 32 x 128 tiles and one matrix; 16 columns, eight waves and one matrix.
MORE = [(32, 0, 16400, 140), (17, 0, 10300, 257), (125, 0, 4050, 200), (27, 0, 10250, 512), (16, 0, 20500, 129),
        (1, 0, 16390, 160), (60, 20, 400, 140), (40, 0, 16500, 135), (16, 0, 70, 140)]

# (offsets, N, K): up to 8 rows a group on average, most of them in one group.
SKEWED = [([0, 3] + [250] * 30 + [256], 100, 140), ([0] * 12 + [200, 205] + [220] * 19, 300, 257),
          ([0] + list(range(0, 32)) + [256], 700, 130), ([7] * 16 + [120] * 17, 1030, 384)]


@pytest.mark.parametrize("rows,groups,N,K", MORE)
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
def test_the_other_kernels_are_exact_on_whole_numbers(lib, rows, groups, N, K, group, zeros):  # noqa: F811
    w4.test_every_tile_is_exact_on_whole_numbers(lib, rows, groups, N, K, group, zeros)


@pytest.mark.parametrize("off,N,K", SKEWED)
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
def test_groups_far_longer_than_their_average(lib, off, N, K, group, zeros):  # noqa: F811
    r = rng(len(off), N, K, group)
    rows, groups = 256, len(off) - 1
    own = [Weights(r, K, N, group, zeros, whole=True) for _ in range(3)]
    ws = [own[g % 3] for g in range(groups)]
    x = torch.from_numpy(r.integers(-3, 4, (rows, K))).to(F16)
    codes, scales, z = stacked(ws)
    C = torch.full((rows, N), -0.125, device="cuda")
    lib.gemm_f16w4f32_grouped(x.cuda(), codes, scales, torch.tensor(off, dtype=torch.int32).cuda(), z, group, C)
    want = torch.full((rows, N), -0.125, dtype=torch.float64)
    for g in range(groups):
        want[off[g]:off[g + 1]] = x[off[g]:off[g + 1]].double() @ ws[g].value
    assert torch.equal(C.cpu().double(), want)


# Groups whose rows lie too far apart for the tiles' offsets: (rows, matrices, N, K).
FAR = (1 << 24) + 8
APART = [(20, 2, 10300, 140), (20, 2, 100, 257), (33, 3, 3000, 140), (44, 5, 2000, 130)]


@pytest.mark.parametrize("rows,groups,N,K", APART)
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
def test_groups_of_rows_far_apart(lib, rows, groups, N, K, group, zeros):  # noqa: F811
    r = rng(rows, groups, N, K, group)
    ws = [Weights(r, K, N, group, zeros, whole=True) for _ in range(groups)]
    off = [0, rows - 2 * (groups - 1)] + [rows - 2 * (groups - 1 - g) for g in range(1, groups)]
    x = torch.from_numpy(r.integers(-3, 4, (rows, K))).to(F16)
    far = torch.empty(FAR * (rows - 1) + K, dtype=F16, device="cuda").as_strided((rows, K), (FAR, 1))
    far.copy_(x)
    codes, scales, z = stacked(ws)
    got = lib.gemm_f16w4f32_grouped(far, codes, scales, torch.tensor(off, dtype=torch.int32).cuda(), z, group)
    want = torch.cat([x[off[g]:off[g + 1]].double() @ ws[g].value for g in range(groups)])
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("N,spare", [(5, 0), (700, 3), (3000, 0)])
def test_groups_without_k_get_zeros(lib, N, spare):  # noqa: F811
    """K = 0: zeros in the rows of a group, the others stay."""
    rows, groups = 50, 4
    C = torch.full((rows + spare, N), 7.0, device="cuda")
    off = torch.tensor([0, 0, 33, 34, rows], dtype=torch.int32).cuda()
    lib.gemm_f16w4f32_grouped(torch.empty(rows + spare, 0, dtype=F16, device="cuda"),
                              torch.empty(groups, 0, N, 64, dtype=torch.uint8, device="cuda"),
                              torch.empty(groups, 0, N, dtype=F16, device="cuda"), off, C=C)
    assert (C[:rows] == 0).all() and (C[rows:] == 7).all()
