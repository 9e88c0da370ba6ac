"""GPU tests of the 4-bit weights, against plain implementations in 64 bits on
the CPU.

Tolerances, from the arithmetic alone (u = 2^-24, half a step of FP32): the
products of FP16 by whole numbers below 256 are exact in FP32; a group's sum and
the sum of the scaled groups are FP32 sums of at most K + K / 32 + 16 terms
together, each step off by at most 2u (a matrix instruction may truncate), and
each scaling by u.  Whole numbers small enough that every sum stays below 2^24,
under scales that are powers of two, have to be exact; so do codes, scales and
zero points."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U2 = 2.0 ** -23
F16, F32 = torch.float16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tiled_dense_gemm_loop_amd as t
    t.load_library()
    return t


def rng(*seed):
    return np.random.default_rng(list(seed))


def normal(r, *shape, scale=1.0):
    return torch.from_numpy(r.standard_normal(shape) * scale).to(F16)


def near(got, want, tol):
    got = got.cpu().double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%d of %d off, the first at %s: got %r, want %r within %r" % (
        int(bad.sum()), bad.numel(), tuple(bad.nonzero()[0].tolist()), float(got[bad][0]), float(want[bad][0]),
        float(tol.expand(got.shape)[bad][0]))


def word_and_bit(k):
    j, q, i = k // 32, k % 32 // 8, k % 8
    return 4 * q + j, 4 * (i // 2) + 16 * (i % 2)


def pack(codes, junk=0):
    """Codes (K x N, 0 .. 15) in the products' layout; `junk` behind K."""
    K, N = codes.shape
    full = np.full((-(-K // 128) * 128, N), junk, dtype=np.uint32)
    full[:K] = codes
    words = np.zeros((full.shape[0] // 128, N, 16), dtype=np.uint32)
    for k in range(128):
        w, bit = word_and_bit(k)
        words[:, :, w] |= full[k::128] << np.uint32(bit)
    return torch.from_numpy(words.view(np.uint8).reshape(-1, N, 64).copy())


def unpack(codes, K):
    words = codes.cpu().contiguous().numpy().view(np.uint32)
    full = np.zeros((words.shape[0] * 128, words.shape[1]), dtype=np.int64)
    for k in range(128):
        w, bit = word_and_bit(k)
        full[k::128] = words[:, :, w] >> np.uint32(bit) & np.uint32(15)
    return full[:K], full[K:]


class Weights:
    """Random 4-bit weights: on the device as the products take them, and their
    values in 64 bits."""

    def __init__(self, r, K, N, group, zeros, whole=False, any_zero=False):
        self.group = group
        q = r.integers(0, 16, (K, N))
        groups = -(-K // group)
        if whole:
            s = 2.0 ** r.integers(-2, 2, (groups, N))
        else:
            s = r.random((groups, N)) + 0.5
        s = torch.from_numpy(s).to(F16)
        z = r.integers(0, 256 if any_zero else 16, (groups, N)) if zeros else np.full((groups, N), 8)
        each = np.arange(K) // group
        self.less = torch.from_numpy((q - z[each]).astype(np.float64))
        self.value = self.less * s.double()[each]
        self.codes = pack(q, junk=15).cuda()
        self.scales = s.cuda()
        self.zeros = torch.from_numpy(z.astype(np.uint8)).cuda() if zeros else None

    @property
    def all(self):
        return self.codes, self.scales, self.zeros


def stacked(ws):
    return (torch.stack([w.codes for w in ws]), torch.stack([w.scales for w in ws]),
            None if ws[0].zeros is None else torch.stack([w.zeros for w in ws]))


def bound(x, value, K):
    return (K + K / 32 + 20) * U2 * (x.double().abs() @ value.abs())


# ------------------------------------------------------------------ quantizing

def quantized(w, group, zeros):
    """scales, zeros, codes by the definition, FP32 step by step."""
    w = w.float().numpy()
    K, N = w.shape
    scales, zs, codes = [], [], []
    with np.errstate(all="ignore"):
        for at in range(0, K, group):
            part = w[at:at + group]
            seen = np.where(np.isnan(part), np.float32(0), part)
            if zeros:
                lo, hi = np.minimum(seen.min(0), np.float32(0)), np.maximum(seen.max(0), np.float32(0))
                s = ((hi - lo) / np.float32(15)).astype(np.float16).astype(np.float32)
                z = np.rint(-lo / s)
                z = np.where((s > 0) & (z >= 0), np.minimum(z, 15), 0).astype(np.float32)
            else:
                s = (np.abs(seen).max(0) / np.float32(7)).astype(np.float16).astype(np.float32)
                z = np.full(N, 8, np.float32)
            q = np.rint(part / s)
            q = np.where((s > 0) & ~np.isnan(q), np.clip(q + z, 0, 15), z)
            scales.append(s), zs.append(z), codes.append(q)
    return np.stack(scales), np.stack(zs), np.concatenate(codes)


def check_quantized(got, w, group, zeros):
    codes, scales, z = got
    ws, wz, wq = quantized(w, group, zeros)
    assert np.array_equal(scales.cpu().float().numpy(), ws)
    assert (z is None) == (not zeros) and (not zeros or np.array_equal(z.cpu().numpy(), wz.astype(np.uint8)))
    q, behind = unpack(codes, w.shape[0])
    assert np.array_equal(q, wq.astype(np.int64)) and not behind.any()


SHAPES = [(1, 1, 32), (1, 65, 128), (31, 3, 32), (32, 64, 32), (33, 130, 64), (128, 257, 128), (129, 40, 96),
          (1000, 77, 64), (384, 33, 96), (500, 64, 128), (700, 19, 1 << 20), (513, 70, 160), (4096, 128, 128),
          (260, 256, 256)]


@pytest.mark.parametrize("K,N,group", SHAPES)
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize(lib, K, N, group, zeros):
    r = rng(K, N, group)
    w = normal(r, K, N, scale=0.1) + (normal(r, 1, N, scale=0.1) if zeros else 0)
    check_quantized(lib.tdg_w4_quantize(w.cuda(), group, zeros), w, group, zeros)


@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_values_that_are_hard(lib, zeros):
    """Zeros, subnormals, the largest values, infinities, NaN, one sign only,
    values between two codes."""
    r = rng(3)
    w = normal(r, 256, 24)
    w[:, 0] = 0
    w[:, 1] = 2.0 ** -24
    w[:, 2] = torch.from_numpy(r.integers(-9, 10, 256) * 2.0 ** -24).to(F16)
    w[:, 3] = 65504
    w[:, 4] = -65504
    w[0::2, 5], w[1::2, 5] = 65504, -65504
    w[7, 6] = float("inf")
    w[200, 7] = float("-inf")
    w[3, 8], w[4, 8] = float("inf"), float("-inf")
    w[9, 9] = float("nan")
    w[:, 10] = float("nan")
    w[:, 11] = w[:, 11].abs() + 1
    w[:, 12] = -w[:, 12].abs() - 1
    w[:, 13] = torch.arange(256).remainder(29).sub(14).to(F16) / 2  # halves of a code
    w[:, 14] = -0.0
    for group in (32, 64, 128, 96, 1024):
        check_quantized(lib.tdg_w4_quantize(w.cuda(), group, zeros), w, group, zeros)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128, 96])
def test_quantize_a_stack_into_strided_outputs(lib, zeros, group):
    r = rng(5, group)
    count, K, N = 3, 300, 50
    w = normal(r, count, K, N)
    groups, blocks = -(-K // group), 3
    wide = torch.full((count, K + 2, N + 9), float("nan"), dtype=F16, device="cuda")
    wide[:, :K, 5:5 + N] = w
    codes = torch.full((count, blocks + 1, N + 3, 64), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((count, groups + 1, N + 3), -3.0, dtype=F16, device="cuda")
    z = torch.full((count, groups + 1, N + 3), 99, dtype=torch.uint8, device="cuda")
    put = (codes[:, :blocks, 2:2 + N], scales[:, :groups, 1:1 + N], z[:, :groups, 3:3 + N])
    got = lib.tdg_w4_quantize(wide[:, :K, 5:5 + N], group, put[2] if zeros else False, put[0], put[1])
    for e in range(count):
        check_quantized([None if t is None else t[e] for t in got], w[e], group, zeros)
    # and nothing beside them
    assert (codes[:, blocks:] == 0x5A).all() and (codes[:, :, :2] == 0x5A).all() and (codes[:, :, 2 + N:] == 0x5A).all()
    assert (scales[:, groups:] == -3).all() and (scales[:, :, 1 + N:] == -3).all() and (scales[:, :, :1] == -3).all()
    assert (z == 99).all() or zeros
    assert (z[:, groups:] == 99).all() and (z[:, :, :3] == 99).all() and (z[:, :, 3 + N:] == 99).all()


@pytest.mark.parametrize("K,N,group", SHAPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_dequantize(lib, K, N, group, zeros, dtype):
    w = Weights(rng(K, N, group, 1), K, N, group, zeros, any_zero=True)
    wide = torch.full((K, N + 3), -7.0, dtype=dtype, device="cuda")
    out = lib.tdg_w4_dequantize(*w.all, K=K, group=group, out=wide[:, 2:2 + N])
    # at most 8 bits by 11: exact in FP32, one rounding to FP16
    assert torch.equal(out.cpu(), w.value.to(dtype))
    assert (wide[:, :2] == -7).all() and (wide[:, 2 + N:] == -7).all()


def test_dequantize_gives_back_what_quantize_rounded(lib):
    w = normal(rng(8), 2, 640, 96)
    codes, scales, _ = lib.tdg_w4_quantize(w.cuda(), 64)
    back = lib.tdg_w4_dequantize(codes, scales, group=64)
    assert back.shape == w.shape and back.dtype == F16
    step = scales.cpu().double().repeat_interleave(64, dim=1)
    # half a step of the code, and half a step of FP16 of at most 8 steps
    assert ((back.cpu().double() - w.double()).abs() <= step * (0.5 + 8 * 2.0 ** -11 + 7 * 2.0 ** -11)).all()


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("wide,apart", [(0, 0), (2, 0), (1, 0), (2, 1), (14, 64)])
def test_stacks_of_many_workgroups(lib, wide, apart, dtype):
    """More workgroups than one round of places, and a last one that is not full; rows and
    matrices that start at whole lines, at multiples of 4 bytes, at odd elements."""
    count, K, N, group = 5, 290, 2034, 64
    ws = [Weights(rng(31, e), K, N, group, True) for e in range(count)]
    ld = N + wide
    stride = K * ld + apart
    flat = torch.full((count * stride,), -7.0, dtype=dtype, device="cuda")
    out = flat.as_strided((count, K, N), (stride, ld, 1))
    lib.tdg_w4_dequantize(*stacked(ws), K=K, group=group, out=out)
    for e in range(count):
        assert torch.equal(out[e].cpu(), ws[e].value.to(dtype))
    assert int((flat == -7.0).sum()) >= count * (K * wide + apart)
    rest = flat.clone()
    rest.as_strided((count, K, N), (stride, ld, 1)).fill_(-7.0)
    assert (rest == -7.0).all()
    if dtype == F16:
        got = lib.tdg_w4_quantize(out, group, True)
        for e in range(count):
            check_quantized([t[e] for t in got], ws[e].value.to(F16), group, True)


# ------------------------------------------------------------------ the product

PRODUCTS = [(1, 1, 1, 32), (1, 16, 32, 32), (1, 17, 33, 64), (2, 100, 128, 128), (3, 64, 129, 32), (15, 33, 500, 96),
            (16, 48, 512, 64), (17, 130, 1000, 128), (31, 65, 96, 96), (33, 16, 2048, 128), (64, 64, 640, 32),
            (65, 127, 257, 64), (100, 31, 1 << 10, 1 << 20), (129, 257, 700, 128), (200, 96, 384, 128),
            (257, 300, 130, 32), (300, 520, 1025, 64), (513, 64, 256, 96), (4, 4096, 1024, 128)]


@pytest.mark.parametrize("M,N,K,group", PRODUCTS)
@pytest.mark.parametrize("zeros", [False, True])
def test_product(lib, M, N, K, group, zeros):
    r = rng(M, N, K, group)
    w, x = Weights(r, K, N, group, zeros), normal(r, M, K)
    got = lib.gemm_f16w4f32(x.cuda(), *w.all, group=group)
    assert got.dtype == F32 and got.shape == (M, N)
    near(got, x.double() @ w.value, bound(x, w.value, K))


@pytest.mark.parametrize("M,N,K,group", PRODUCTS)
def test_product_of_whole_numbers_is_exact(lib, M, N, K, group):
    r = rng(M, N, K, group, 2)
    w = Weights(r, K, N, group, True, whole=True)
    x = torch.from_numpy(r.integers(-3, 4, (M, K))).to(F16)
    got = lib.gemm_f16w4f32(x.cuda(), *w.all, group=group)
    assert torch.equal(got.cpu().double(), x.double() @ w.value)


@pytest.mark.parametrize("M", [1, 20, 150])
@pytest.mark.parametrize("K,group", [(130, 32), (250, 128), (384, 64)])
def test_product_of_strided_operands(lib, M, K, group):
    """Rows, columns and blocks inside larger arrays that hold NaN and other
    codes, rows off any grid, and a C whose surroundings stay."""
    r = rng(M, K)
    N = 37
    w, x = Weights(r, K, N, group, True), normal(r, M, K)
    wide = torch.full((M, K + 7), float("nan"), dtype=F16, device="cuda")
    wide[:, 3:3 + K] = x
    codes = torch.full((w.codes.shape[0], N + 4, 64), 0xFF, dtype=torch.uint8, device="cuda")
    codes[:, 1:1 + N] = w.codes
    scales = torch.full((w.scales.shape[0], N + 4), float("nan"), dtype=F16, device="cuda")
    scales[:, 2:2 + N] = w.scales
    zeros = torch.full((w.scales.shape[0], N + 4), 255, dtype=torch.uint8, device="cuda")
    zeros[:, 3:3 + N] = w.zeros
    C = torch.full((M + 1, N + 6), -5.0, device="cuda")
    lib.gemm_f16w4f32(wide[:, 3:3 + K], codes[:, 1:1 + N], scales[:, 2:2 + N], zeros[:, 3:3 + N], group,
                      C[:M, 4:4 + N])
    near(C[:M, 4:4 + N], x.double() @ w.value, bound(x, w.value, K))
    C[:M, 4:4 + N] = -5
    assert (C == -5).all()


def at_page_end(t):
    """t on the device, its last byte the last of a 4 KiB page; NaN behind."""
    bytes_ = t.numel() * t.element_size()
    buf = torch.full(((bytes_ + 8192) // t.element_size(),), float("nan"), dtype=t.dtype, device="cuda")
    skip = (-(buf.data_ptr() + bytes_)) % 4096 // t.element_size()
    v = buf[skip:skip + t.numel()].view(t.shape)
    return v.copy_(t)


@pytest.mark.parametrize("M,K", [(1, 129), (3, 1001), (70, 517), (200, 255)])
def test_rows_that_end_with_their_page(lib, M, K):
    r = rng(M, K)
    w, x = Weights(r, K, 48, 64, False), normal(r, M, K)
    near(lib.gemm_f16w4f32(at_page_end(x), *w.all, group=64), x.double() @ w.value, bound(x, w.value, K))


def test_product_values_that_are_hard(lib):
    """Subnormal and largest elements, zero points far from the codes, scales
    of 0, a scale of infinity in one column alone, NaN and infinities in rows
    that stay in their rows."""
    r = rng(11)
    M, N, K = 40, 20, 256
    w, x = Weights(r, K, N, 64, True, any_zero=True), normal(r, M, K)
    x[1] *= 2.0 ** -18
    x[2] = 65504
    x[3] = torch.from_numpy(r.integers(-9, 10, K) * 2.0 ** -24).to(F16)
    want, tol = x.double() @ w.value, bound(x, w.value, K)
    near(lib.gemm_f16w4f32(x.cuda(), *w.all, group=64), want, tol)
    y = x.clone()
    y[5, 7] = float("nan")
    y[6, 9] = float("inf")
    scales = w.scales.clone()
    scales[1, 4] = float("inf")
    scales[2, 5] = 0
    got = lib.gemm_f16w4f32(y.cuda(), w.codes, scales, w.zeros, 64).cpu()
    assert got[5].isnan().all() and not got[6].isfinite().any()
    rows = [i for i in range(M) if i not in (5, 6)]
    cols = [i for i in range(N) if i not in (4, 5)]
    near(got[rows][:, cols], want[rows][:, cols], tol[rows][:, cols])
    assert not got[rows][:, 4].isfinite().any()
    part = w.value.clone()
    part[128:192, 5] = 0
    near(got[rows][:, 5:6], (x.double() @ part)[rows][:, 5:6], tol[rows][:, 5:6])


def test_empty_products(lib):
    w = Weights(rng(1), 64, 5, 32, False)
    none = torch.empty(0, 64, dtype=F16, device="cuda")
    assert lib.gemm_f16w4f32(none, *w.all, group=32).shape == (0, 5)
    C = torch.full((3, 5), 4.0, device="cuda")
    codes, scales = (torch.empty(0, 5, 64, dtype=torch.uint8, device="cuda"), torch.empty(0, 5, dtype=F16, device="cuda"))
    lib.gemm_f16w4f32(torch.empty(3, 0, dtype=F16, device="cuda"), codes, scales, C=C)
    assert (C == 0).all()


@pytest.mark.parametrize("M", [3, 130])
def test_rows_more_than_32_bits_apart(lib, M):
    """A's and C's rows, and the blocks of codes, past 2^32 bytes."""
    r = rng(M, 9)
    K, N, group = 300, 24, 64
    w, x = Weights(r, K, N, group, False), normal(r, M, K)
    far = (5 << 30) // 2 // (M - 1) + 8
    big = torch.empty(far * (M - 1) + K, dtype=F16, device="cuda")
    rows = big.as_strided((M, K), (far, 1))
    rows.copy_(x)
    apart = (5 << 30) // 2 // 64 + 3
    codes = torch.empty((apart * 2 + N) * 64, dtype=torch.uint8, device="cuda").as_strided((3, N, 64), (apart * 64, 64, 1))
    codes.copy_(w.codes)
    C = torch.empty(far * (M - 1) + N, device="cuda").as_strided((M, N), (far, 1))
    lib.gemm_f16w4f32(rows, codes, w.scales, group=group, C=C)
    near(C, x.double() @ w.value, bound(x, w.value, K))


def test_tiles_whose_rows_pass_32_bits(lib):
    """Rows near enough for the LDS tiles' offsets, 6 GB in all."""
    r = rng(10)
    M, K, N, far = 400, 140, 3000, 8 << 20
    w, x = Weights(r, K, N, 64, False), normal(r, M, K)
    rows = torch.empty(far * (M - 1) + K, dtype=F16, device="cuda").as_strided((M, K), (far, 1))
    rows.copy_(x)
    near(lib.gemm_f16w4f32(rows, *w.all, group=64), x.double() @ w.value, bound(x, w.value, K))


@pytest.mark.parametrize("group", [64, 96])
def test_quantizing_rows_that_pass_32_bits(lib, group):
    K, N, far = 200, 40, 16 << 20
    w = normal(rng(group), K, N)
    rows = torch.empty(far * (K - 1) + N, dtype=F16, device="cuda").as_strided((K, N), (far, 1))
    rows.copy_(w)
    got = lib.tdg_w4_quantize(rows, group, True)
    check_quantized(got, w, group, True)
    out = torch.empty(far * (K - 1) + N, dtype=F16, device="cuda").as_strided((K, N), (far, 1))
    lib.tdg_w4_dequantize(*got, K=K, group=group, out=out)
    assert torch.equal(out.cpu(), lib.tdg_w4_dequantize(*got, K=K, group=group).cpu())


# ------------------------------------------------------------------ the experts' products

GROUPED = [(1, 1, 1, 1, 32), (4, 9, 33, 100, 64), (64, 32, 48, 256, 128), (37, 3, 130, 257, 96), (333, 9, 61, 1000, 32),
           (200, 2, 64, 128, 128), (1000, 5, 257, 140, 64), (700, 40, 16, 513, 128), (2, 1024, 16, 32, 32),
           (1500, 6, 300, 256, 128)]


def offsets_of(r, rows, groups):
    cuts = np.sort(r.integers(0, rows + 1, groups - 1)) if groups > 1 else np.zeros(0, np.int64)
    return [0] + cuts.tolist() + [rows]


@pytest.mark.parametrize("rows,groups,N,K,group", GROUPED)
@pytest.mark.parametrize("zeros", [False, True])
def test_grouped(lib, rows, groups, N, K, group, zeros):
    r = rng(rows, groups, N, K)
    off = offsets_of(r, rows, groups)
    ws = [Weights(r, K, N, group, zeros) for _ in range(min(groups, 9))]
    ws = [ws[g % len(ws)] for g in range(groups)]
    spare = 5
    x = normal(r, rows + spare, K)
    x[rows:] = float("nan")
    C = torch.full((rows + spare, N), -5.0, device="cuda")
    codes, scales, z = stacked(ws)
    lib.gemm_f16w4f32_grouped(x.cuda(), codes, scales, torch.tensor(off, dtype=torch.int32).cuda(), z, group, C)
    want = torch.full((rows + spare, N), -5.0, dtype=torch.float64)
    tol = torch.zeros(rows + spare, N, dtype=torch.float64)
    for g in range(groups):
        lo, hi = off[g], off[g + 1]
        want[lo:hi] = x[lo:hi].double() @ ws[g].value
        tol[lo:hi] = bound(x[lo:hi], ws[g].value, K)
    near(C, want, tol)


@pytest.mark.parametrize("rows", [20, 400])
def test_grouped_offsets_that_leave_rows_out_or_point_outside(lib, rows):
    """Rows before the first and behind the last offset stay; offsets are
    clamped to the rows; a matrix without rows may hold anything."""
    r = rng(rows, 77)
    K, N, group = 160, 40, 32
    ws = [Weights(r, K, N, group, False) for _ in range(5)]
    codes, scales, _ = stacked(ws)
    scales[1] = float("nan")
    x = normal(r, rows, K)
    third = rows // 3
    off = [2, third, third, 2 * third, rows - 3, rows - 3]
    C = torch.full((rows, N), -5.0, device="cuda")
    lib.gemm_f16w4f32_grouped(x.cuda(), codes, scales, torch.tensor(off, dtype=torch.int32).cuda(), group=group, C=C)
    want, tol = torch.full((rows, N), -5.0, dtype=torch.float64), torch.zeros(rows, N, dtype=torch.float64)
    for g in (0, 2, 3):
        lo, hi = off[g], off[g + 1]
        want[lo:hi], tol[lo:hi] = x[lo:hi].double() @ ws[g].value, bound(x[lo:hi], ws[g].value, K)
    near(C, want, tol)
    off = [-(2 ** 31), third, third, third, rows - 3, 2 ** 31 - 1]
    C.fill_(-5.0)
    lib.gemm_f16w4f32_grouped(x.cuda(), codes, scales, torch.tensor(off, dtype=torch.int32).cuda(), group=group, C=C)
    for g, lo, hi in ((0, 0, third), (3, third, rows - 3), (4, rows - 3, rows)):
        want[lo:hi], tol[lo:hi] = x[lo:hi].double() @ ws[g].value, bound(x[lo:hi], ws[g].value, K)
    near(C, want, tol)


@pytest.mark.parametrize("rows", [24, 500])
def test_grouped_offsets_that_do_not_ascend(lib, rows):
    """Each element of a row is one of its groups' products, or stays (column
    tiles run in any order, so a row may hold several groups')."""
    r = rng(rows, 78)
    K, N, group = 128, 33, 64
    ws = [Weights(r, K, N, group, False) for _ in range(6)]
    codes, scales, _ = stacked(ws)
    x = normal(r, rows, K)
    for off in ([0, rows, 5, rows, 0, 0, rows], [rows, 0, rows, 0, rows, 0, rows], [7, 7, 3, 1, -4, rows + 9, 2]):
        C = torch.full((rows, N), -5.0, device="cuda")
        lib.gemm_f16w4f32_grouped(x.cuda(), codes, scales, torch.tensor(off, dtype=torch.int32).cuda(), group=group,
                                  C=C)
        got, fits = C.cpu().double(), C.cpu() == -5
        for w in ws:
            fits |= (got - x.double() @ w.value).abs() <= bound(x, w.value, K)
        assert fits.all()


def test_grouped_one_matrix_for_all_groups(lib):
    r = rng(4)
    w, x = Weights(r, 200, 30, 96, True), normal(r, 50, 200)
    codes, scales, z = (t.expand((3,) + t.shape) for t in w.all)
    off = torch.tensor([0, 10, 10, 50], dtype=torch.int32).cuda()
    near(lib.gemm_f16w4f32_grouped(x.cuda(), codes, scales, off, z, 96), x.double() @ w.value, bound(x, w.value, 200))


# ------------------------------------------------------------------ every tile

# (rows, matrices or 0 for the plain product, N, K): 128 x 512, 64 x 256, 64 x 128,
# 32 x 128 and 32 x 64 tiles and the kernels of few rows, by the rule that picks them.
TILES = [(1000, 0, 3500, 130), (450, 0, 3900, 257), (1030, 0, 13000, 130), (1100, 0, 6000, 155), (700, 0, 3000, 256), (70, 0, 8200, 300), (130, 0, 3900, 200),
         (40, 0, 4100, 129), (24, 0, 4100, 384), (9, 0, 300, 8200), (2100, 2, 6600, 70), (2000, 6, 3300, 257),
         (1000, 5, 2000, 128), (700, 40, 800, 200), (300, 20, 300, 391), (150, 30, 500, 140)]


@pytest.mark.parametrize("rows,groups,N,K", TILES)
@pytest.mark.parametrize("group", [32, 64, 128, 96])
@pytest.mark.parametrize("zeros", [False, True])
def test_every_tile_is_exact_on_whole_numbers(lib, rows, groups, N, K, group, zeros):
    """Whole numbers against 64 bits; and the same with LDS full of NaN first,
    which a read of a buffer that is not filled yet would show."""
    r = rng(rows, groups, N, K, group)
    ws = [Weights(r, K, N, group, zeros, whole=True) for _ in range(min(groups, 3) or 1)]
    x = torch.from_numpy(r.integers(-3, 4, (rows, K))).to(F16)
    X = x.cuda()
    if groups:
        ws = [ws[g % len(ws)] for g in range(groups)]
        off = offsets_of(r, rows, groups)
        codes, scales, z = stacked(ws)
        d = torch.tensor(off, dtype=torch.int32).cuda()
        run = lambda: lib.gemm_f16w4f32_grouped(X, codes, scales, d, z, group)  # noqa: E731
        want = torch.cat([x[off[g]:off[g + 1]].double() @ ws[g].value for g in range(groups)])
    else:
        run = lambda: lib.gemm_f16w4f32(X, *ws[0].all, group=group)  # noqa: E731
        want = x.double() @ ws[0].value
    assert torch.equal(run().cpu().double(), want)
    old = lib.tdg_set_debug_flags(lib.TDG_DEBUG_POISON_LDS)
    try:
        assert torch.equal(run().cpu().double(), want)
    finally:
        lib.tdg_set_debug_flags(old)


@pytest.mark.parametrize("M,N,K", [(70, 8200, 261), (700, 3000, 133), (1100, 6000, 100), (1030, 13000, 135)])
def test_tiles_of_strided_rows_that_end_with_their_page(lib, M, N, K):
    """Rows off any grid, NaN between them and behind the last; C's
    surroundings stay."""
    r = rng(M, N, K)
    w, x = Weights(r, K, N, 64, True), normal(r, M, K)
    wide = torch.full((M, K + 3), float("nan"), dtype=F16)
    wide[:, 3:] = x
    C = torch.full((M + 1, N + 2), -5.0, device="cuda")
    lib.gemm_f16w4f32(at_page_end(wide)[:, 3:], *w.all, group=64, C=C[:M, 1:1 + N])
    near(C[:M, 1:1 + N], x.double() @ w.value, bound(x, w.value, K))
    C[:M, 1:1 + N] = -5
    assert (C == -5).all()


# ------------------------------------------------------------------ together, streams, graphs

def test_a_routed_layer_with_quantized_experts(lib):
    """Quantize, plan, dispatch, both products and combine, as they are used;
    against 64 bits with the quantized values."""
    r = rng(21)
    T, k, E, H, I = 50, 2, 6, 256, 192
    up, down = normal(r, E, H, 2 * I, scale=H ** -0.5), normal(r, E, I, H, scale=I ** -0.5)
    x = normal(r, T, H)
    ids = torch.from_numpy(r.integers(0, E, (T, k))).to(torch.int32)
    ids[-3:] = -1
    wt = torch.from_numpy(r.random((T, k))).to(F32)
    q_up, q_down = lib.tdg_w4_quantize(up.cuda(), 64, True), lib.tdg_w4_quantize(down.cuda(), 32)
    offsets, order, slots = lib.tdg_route_plan(ids.cuda(), E)
    xs = lib.tdg_rows_dispatch(x.cuda(), slots, out=torch.zeros(T * k, H, dtype=F16, device="cuda"))
    both = lib.gemm_f16w4f32_grouped(xs, q_up[0], q_up[1], offsets, q_up[2], 64,
                                     C=torch.zeros(T * k, 2 * I, device="cuda"))
    h = (torch.nn.functional.silu(both[:, :I]) * both[:, I:]).half()
    z = lib.gemm_f16w4f32_grouped(h, q_down[0], q_down[1], offsets, q_down[2], 32,
                                  C=torch.zeros(T * k, H, device="cuda"))
    y = lib.tdg_rows_combine(z, slots, wt.cuda())
    vu = lib.tdg_w4_dequantize(*q_up, K=H, group=64, out_dtype=F32).cpu().double()
    vd = lib.tdg_w4_dequantize(*q_down, K=I, group=32, out_dtype=F32).cpu().double()
    want, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T - 3):
        for j in range(k):
            e = int(ids[t, j])
            b = x[t].double() @ vu[e]
            tb = 2 * H * U2 * (x[t].double().abs() @ vu[e].abs())
            g, u = b[:I], b[I:]
            h64 = g * torch.sigmoid(g) * u
            # silu's slope is below 1.1; h is rounded to FP16 once
            th = 1.1 * (tb[:I] * u.abs() + g.abs() * tb[I:] + tb[:I] * tb[I:]) + h64.abs() * 2.0 ** -10.9 + 2.0 ** -24
            want[t] += wt[t, j].double() * (h64 @ vd[e])
            tol[t] += float(wt[t, j]) * (th @ vd[e].abs() + 2 * I * U2 * (h64.abs() @ vd[e].abs()) + 1e-6)
    near(y, want, tol)


def test_on_another_stream_and_in_a_graph(lib):
    """Calls follow torch's current stream, and a captured run of them gives the
    eager results again on new inputs."""
    r = rng(31)
    K, N, M = 384, 96, 18
    ws = [Weights(r, K, N, 64, True) for _ in range(3)]
    codes, scales, zeros = stacked(ws)
    off = torch.tensor([0, 7, 7, M], dtype=torch.int32).cuda()
    xs = [normal(r, M, K).cuda() for _ in range(4)]
    big = [normal(r, 300, K).cuda() for _ in range(4)]

    def run(x, b, w):
        q = lib.tdg_w4_quantize(w, 64, True)
        return (lib.gemm_f16w4f32(x, *ws[0].all, group=64), lib.gemm_f16w4f32(b, *ws[1].all, group=64),
                lib.gemm_f16w4f32_grouped(x, codes, scales, off, zeros, 64), q[0], q[1], q[2],
                lib.tdg_w4_dequantize(*q, K=K, group=64))

    weights = [normal(r, K, N).cuda() for _ in range(4)]
    want = [run(*a) for a in zip(xs, big, weights)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run(xs[0], big[0], weights[0])
    side.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want[0]))
    x, b, w = xs[0].clone(), big[0].clone(), weights[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(x, b, w)
    for i in (1, 2, 3, 1):
        x.copy_(xs[i]), b.copy_(big[i]), w.copy_(weights[i])
        graph.replay()
        eager = run(xs[i], big[i], weights[i])
        torch.cuda.synchronize()
        assert all(torch.equal(g, w_) for g, w_ in zip(got, want[i]))
        assert all(torch.equal(g, w_) for g, w_ in zip(eager, want[i]))


def test_wrong_shapes_are_refused(lib):
    w = Weights(rng(1), 256, 8, 64, True)
    x = torch.zeros(4, 256, dtype=F16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    stack = tuple(t[None].expand((2,) + t.shape).contiguous() for t in w.all)
    ok = lib.gemm_f16w4f32(x, *w.all, group=64)
    assert ok.shape == (4, 8)
    for call in (lambda: lib.gemm_f16w4f32(x, *w.all, group=128), lambda: lib.gemm_f16w4f32(x, *w.all, group=16),
                 lambda: lib.gemm_f16w4f32(x[:, :100], *w.all, group=64),
                 lambda: lib.gemm_f16w4f32(x, w.codes[:, :7], w.scales, w.zeros, 64),
                 lambda: lib.gemm_f16w4f32(x, w.codes.view(2, 4, 128), w.scales, w.zeros, 64),
                 lambda: lib.gemm_f16w4f32(x, w.codes, w.scales, w.zeros.t(), 64),
                 lambda: lib.gemm_f16w4f32(x, w.codes.cpu(), w.scales, w.zeros, 64),
                 lambda: lib.gemm_f16w4f32(x, *w.all, group=64, C=torch.zeros(4, 9, device="cuda")),
                 lambda: lib.gemm_f16w4f32_grouped(x, stack[0], stack[1], off[:2], stack[2], 64),
                 lambda: lib.gemm_f16w4f32_grouped(x, stack[0], stack[1][:1], off, stack[2], 64),
                 lambda: lib.gemm_f16w4f32_grouped(x, w.codes, w.scales, off, w.zeros, 64),
                 lambda: lib.tdg_w4_dequantize(*w.all, K=128, group=64),
                 lambda: lib.tdg_w4_dequantize(*w.all, K=256, group=64, out=torch.zeros(255, 8, device="cuda")),
                 lambda: lib.tdg_w4_quantize(x, 24), lambda: lib.tdg_w4_quantize(x, 64, codes=w.codes)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lib.gemm_f16w4f32(x, w.codes.char(), w.scales, w.zeros, 64),
                 lambda: lib.gemm_f16w4f32(x, w.codes, w.scales.float(), w.zeros, 64),
                 lambda: lib.gemm_f16w4f32(x, w.codes, w.scales, w.zeros.int(), 64),
                 lambda: lib.gemm_f16w4f32(x, *w.all, group=64, C=x[:, :8])):
        with pytest.raises(TypeError):
            call()
