"""GPU tests of the layer of experts for a few tokens, against a plain
implementation in 64 bits on the CPU.

Tolerances, from the arithmetic alone (u = 2^-24, half a step of FP32): a sum of
n products in FP32 is off by at most (n + 8) * 2u * sum |a b| (a matrix
instruction may truncate); silu's slope is below 1.1 in size, and its own
arithmetic (an exponential within an ulp or two, a sum, a quotient, a product)
is off by less than 16u; y adds a rounding for each of top_k products and sums,
and one to its type."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U2 = 2.0 ** -23
F16, F32, F64 = torch.float16, torch.float32, torch.float64


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


def layer64(x, ids, weights, up, down, dtype):
    """y and how far it may be off."""
    T, k = ids.shape
    E, inner, cols = down.shape
    y, tol = torch.zeros(T, cols, dtype=F64), torch.zeros(T, cols, dtype=F64)
    size = torch.zeros(T, cols, dtype=F64)
    for e in range(E):
        for t, j in (ids == e).nonzero().tolist():
            a, w = x[t].double(), 1.0 if weights is None else float(weights[t, j])
            b = a @ up[e].double()
            tb = (cols + 8) * U2 * (a.abs() @ up[e].double().abs())
            g, u, tg, tu = b[:inner], b[inner:], tb[:inner], tb[inner:]
            silu = g * torch.sigmoid(g)
            h = silu * u
            th = 1.1 * tg * (u.abs() + tu) + silu.abs() * tu + 8 * U2 * h.abs() + 2.0 ** -120
            d = down[e].double()
            z = h @ d
            tz = (inner + 8) * U2 * (h.abs() @ d.abs()) + th @ d.abs() * (1 + inner * U2)
            y[t] += w * z
            tol[t] += abs(w) * tz
            size[t] += abs(w) * z.abs()
    tol += (k + 1) * U2 * size + (y.abs() * 2.0 ** -11 + 2.0 ** -25 if dtype == F16 else y.abs() * 2.0 ** -24)
    return y, tol


def near(got, want, tol):
    got = got.cpu().double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%d of %d off, the first at %s: got %r, want %r within %r" % (
        int(bad.sum()), bad.numel(), tuple(bad.nonzero()[0].tolist()), float(got[bad][0]), float(want[bad][0]),
        float(tol[bad][0]))


def problem(r, T, k, E, cols, inner, distinct=True):
    x = normal(r, T, cols)
    up, down = normal(r, E, cols, 2 * inner, scale=cols ** -0.5), normal(r, E, inner, cols, scale=inner ** -0.5)
    if distinct:
        ids = np.stack([r.permutation(E)[:k] for _ in range(T)])
    else:
        ids = r.integers(0, E, (T, k))
    return x, torch.from_numpy(ids).to(torch.int32), torch.from_numpy(r.random((T, k))).to(F32), up, down


SIZES = [(1, 1, 1, 1, 1), (1, 8, 8, 64, 32), (1, 2, 16, 7, 5), (2, 1, 4, 8, 8), (3, 2, 3, 33, 9), (5, 8, 32, 256, 96),
         (7, 3, 5, 100, 70), (8, 1, 128, 130, 65), (16, 4, 8, 64, 129), (17, 2, 2, 40, 24), (33, 2, 8, 257, 63),
         (64, 1, 1, 72, 40), (64, 8, 16, 128, 64), (1, 8, 128, 1024, 384), (64, 2, 3, 31, 200), (40, 8, 64, 63, 17),
         (1, 32, 40, 48, 16), (64, 32, 32, 16, 16)]


@pytest.mark.parametrize("T,k,E,cols,inner", SIZES)
@pytest.mark.parametrize("dtype", [F16, F32])
def test_layer(lib, T, k, E, cols, inner, dtype):
    p = problem(rng(T, k, E, cols, inner), T, k, E, cols, inner)
    got = lib.tdg_expert_layer(*(t.cuda() for t in p), out_dtype=dtype)
    assert got.dtype == dtype and got.shape == (T, cols)
    near(got, *layer64(*p, dtype))


# Every way to cut the work: k of the up product in two and four parts beside both
# shapes of down, k of down in two, more rows than one tile with each.
CUTS = [(3, 2, 8, 600, 200), (2, 2, 8, 1100, 600), (20, 2, 16, 1600, 520), (20, 2, 16, 1600, 500), (40, 1, 2, 1030, 100),
        (64, 8, 64, 1100, 130), (1, 1, 1, 4096, 1100), (50, 1, 2, 520, 700), (33, 2, 8, 2050, 300), (2, 2, 4, 1025, 129),
        (5, 2, 4, 1024, 2048)]  # (the last: as much LDS as any)


@pytest.mark.parametrize("T,k,E,cols,inner", CUTS)
def test_every_cut_of_the_work(lib, T, k, E, cols, inner):
    p = problem(rng(T, k, E, cols, inner), T, k, E, cols, inner)
    p = p[:1] + (torch.where(p[1] == 0, -1, p[1]).to(torch.int32) if T > 20 else p[1],) + p[2:]
    need = lib.tdg_expert_layer_workspace(T, k, E, cols, inner)
    work = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN, wherever it is read
    got = lib.tdg_expert_layer(*(t.cuda() for t in p), out_dtype=F32, workspace=work)
    near(got, *layer64(*p, F32))


def test_no_inner_columns_give_zeros(lib):
    x, ids, w, up, down = problem(rng(2), 3, 2, 4, 20, 8)
    y = torch.full((3, 20), 5.0, device="cuda")
    lib.tdg_expert_layer(x.cuda(), ids.cuda(), w.cuda(), up[:, :, :0].cuda(), down[:, :0].cuda(), out=y)
    assert (y == 0).all()


@pytest.mark.parametrize("T,k,E", [(1, 6, 2), (30, 3, 2), (64, 32, 2), (20, 4, 100)])
def test_the_same_expert_twice_and_ids_outside(lib, T, k, E):
    r = rng(T, k, E)
    x, ids, w, up, down = problem(r, T, k, E, 72, 40, distinct=False)
    drop = torch.from_numpy(r.random((T, k)) < 0.3)
    ids[drop] = torch.from_numpy(r.choice([-1, E, 2 ** 31 - 1, -2 ** 31], int(drop.sum()))).to(torch.int32)
    if T > 1:
        ids[-1] = -1  # a token without an expert
    y = torch.full((T, 72), float("nan"), device="cuda")
    lib.tdg_expert_layer(x.cuda(), ids.cuda(), w.cuda(), up.cuda(), down.cuda(), out=y)
    near(y, *layer64(x, ids, w, up, down, F32))
    assert T == 1 or (y[-1] == 0).all()


def test_without_weights_and_without_any_expert(lib):
    x, ids, w, up, down = problem(rng(6), 9, 3, 5, 50, 20)
    dev = [t.cuda() for t in (x, ids, up, down)]
    near(lib.tdg_expert_layer(dev[0], dev[1], None, dev[2], dev[3]), *layer64(x, ids, None, up, down, F16))
    out = lib.tdg_expert_layer(dev[0], torch.full_like(dev[1], -1), None, dev[2], dev[3])
    assert (out == 0).all()


def test_nothing_of_an_expert_that_a_token_did_not_pick(lib):
    """Matrices of NaN and infinities reach the tokens that name them, alone."""
    r = rng(12)
    T, E, cols, inner = 20, 6, 96, 40
    x, ids, w, up, down = problem(r, T, 2, E, cols, inner)
    ids[ids == 2] = 3
    ids[ids == 4] = 5
    ids[4, 0], ids[11, 1] = 2, 4
    up[2], down[4] = float("nan"), float("inf")
    x[7] = float("inf")  # a row of infinities stays a row
    up[0], down[0] = float("nan"), float("nan")
    ids[ids == 0] = 1
    got = lib.tdg_expert_layer(*(t.cuda() for t in (x, ids, w, up, down)), out_dtype=F32).cpu()
    rest = [t for t in range(T) if t not in (4, 7, 11)]
    y, tol = layer64(x[rest], ids[rest], w[rest], up, down, F32)
    near(got[rest], y, tol)
    assert got[4].isnan().all() and not got[7].isfinite().any() and not got[11].isfinite().any()


@pytest.mark.parametrize("T,k,E,cols,inner", [(2, 2, 4, 70, 21), (40, 2, 3, 45, 33), (1, 1, 2, 6, 3)])
def test_strided_operands(lib, T, k, E, cols, inner):
    """Rows inside larger arrays of NaN, at odd offsets; y's surroundings stay."""
    r = rng(T, cols)
    p = problem(r, T, k, E, cols, inner)
    x, ids, w, up, down = p

    def inside(t, pad, fill):
        shape = list(t.shape)
        shape[-1] += pad
        shape[-2] += 1
        buf = torch.full(shape, fill, dtype=t.dtype, device="cuda")
        v = buf[..., :t.shape[-2], pad // 2:pad // 2 + t.shape[-1]]
        v.copy_(t)
        return v

    nan = float("nan")
    y = torch.full((T + 1, cols + 5), -3.0, device="cuda")
    lib.tdg_expert_layer(inside(x, 3, nan), inside(ids, 5, 0), inside(w, 4, nan), inside(up, 7, nan),
                         inside(down, 5, nan), out=y[:T, 2:2 + cols])
    near(y[:T, 2:2 + cols], *layer64(*p, F32))
    y[:T, 2:2 + cols] = -3
    assert (y == -3).all()


def at_page_end(t):
    bytes_ = t.numel() * t.element_size()
    buf = torch.full(((bytes_ + 8192) // t.element_size(),), float("nan"), dtype=t.dtype, device="cuda")
    skip = (-(buf.data_ptr() + bytes_)) % 4096 // t.element_size()
    return buf[skip:skip + t.numel()].view(t.shape).copy_(t)


@pytest.mark.parametrize("cols,inner", [(65, 33), (40, 7), (31, 129)])
def test_operands_that_end_with_their_page(lib, cols, inner):
    p = problem(rng(cols, inner), 5, 2, 3, cols, inner)
    x, ids, w, up, down = p
    got = lib.tdg_expert_layer(at_page_end(x), ids.cuda(), w.cuda(), at_page_end(up), at_page_end(down))
    near(got, *layer64(*p, F16))


def test_large_and_small_gates(lib):
    """Gates whose exponential overflows and vanishes, elements of h far apart
    in size: each column of down keeps what only a small one reaches."""
    T, E, cols, inner = 6, 2, 64, 32
    r = rng(13)
    x, ids, w, up, down = problem(r, T, 1, E, cols, inner)
    scale = torch.from_numpy(2.0 ** r.integers(-14, 9, (1, 1, 2 * inner))).to(F16)
    up = (up.float() * scale.float()).half()
    down = torch.zeros(E, inner, cols, dtype=F16)
    for i in range(inner):  # one element of h each
        down[:, i, 2 * i] = 1
    got = lib.tdg_expert_layer(*(t.cuda() for t in (x, ids, w, up, down)), out_dtype=F32)
    near(got, *layer64(x, ids, w, up, down, F32))


def test_matrices_more_than_32_bits_apart(lib):
    r = rng(14)
    T, k, E, cols, inner = 4, 2, 3, 40, 24
    x, ids, w, up, down = problem(r, T, k, E, cols, inner)
    apart = (5 << 30) // 2

    def far(t):
        big = torch.empty(apart * (E - 1) + t[0].numel(), dtype=F16, device="cuda")
        v = big.as_strided(t.shape, (apart, t.shape[2], 1))
        return v.copy_(t)

    got = lib.tdg_expert_layer(x.cuda(), ids.cuda(), w.cuda(), far(up), far(down))
    near(got, *layer64(x, ids, w, up, down, F16))


def test_the_same_values_as_the_sorted_path(lib):
    """The layer beside the plan, the grouped products and the combine: the
    same 64-bit values, each within its own bound (their h is rounded to FP16)."""
    r = rng(15)
    T, k, E, H, I = 24, 2, 5, 128, 96
    x, ids, w, up, down = problem(r, T, k, E, H, I)
    dev = [t.cuda() for t in (x, ids, w, up, down)]
    y, tol = layer64(x, ids, w, up, down, F32)
    near(lib.tdg_expert_layer(*dev, out_dtype=F32), y, tol)
    offsets, order, slots = lib.tdg_route_plan(dev[1], E)
    both = lib.gemm_f16f32_grouped(lib.tdg_rows_dispatch(dev[0], slots), dev[3], offsets)
    h = (torch.nn.functional.silu(both[:, :I]) * both[:, I:]).half()
    z = lib.gemm_f16f32_grouped(h, dev[4], offsets)
    coarse = torch.zeros_like(tol)
    for t in range(T):
        for j in range(k):
            b = x[t].double() @ up[ids[t, j]].double()
            h64 = (b[:I] * torch.sigmoid(b[:I]) * b[I:]).abs()
            coarse[t] += w[t, j].double() * ((h64 * 2.0 ** -10.9 + 2.0 ** -24) @ down[ids[t, j]].double().abs())
    near(lib.tdg_rows_combine(z, slots, dev[2]), y, tol + coarse)


def test_on_other_streams_and_in_graphs(lib):
    """Two calls at once with a workspace each; a captured call, replayed on new
    inputs, gives the eager results; the same bits from run to run."""
    r = rng(16)
    T, k, E, cols, inner = 12, 4, 16, 192, 72
    ps = [problem(rng(16, i), T, k, E, cols, inner) for i in range(4)]
    dev = [[t.cuda() for t in p] for p in ps]
    want = [lib.tdg_expert_layer(*d) for d in dev]
    for d, p, y in zip(dev, ps, want):
        near(y, *layer64(*p, F16))
        assert torch.equal(y, lib.tdg_expert_layer(*d))
    need = lib.tdg_expert_layer_workspace(T, k, E, cols, inner)
    side = [torch.cuda.Stream() for _ in range(2)]
    work = [torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i, s in enumerate(side):
        with torch.cuda.stream(s):
            got.append([lib.tdg_expert_layer(*dev[i], workspace=work[i]) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    held = [t.clone() for t in dev[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lib.tdg_expert_layer(*held, workspace=work[0])
    for i in (1, 2, 3, 1):
        for h, t in zip(held, dev[i]):
            h.copy_(t)
        graph.replay()
        eager = lib.tdg_expert_layer(*dev[(i + 1) % 4])
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]) and torch.equal(eager, want[(i + 1) % 4])
    # and one whose first product is cut, so that the second joins its parts
    cut = [[t.cuda() for t in problem(rng(17, i), 3, 2, 8, 1030, 200)] for i in range(2)]
    eager = [lib.tdg_expert_layer(*c) for c in cut]
    held = [t.clone() for t in cut[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lib.tdg_expert_layer(*held)
    for i in (1, 0, 1):
        for h, t in zip(held, cut[i]):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])
    # one workspace for calls of several sizes that follow each other
    small = problem(r, 2, 3, 16, 192, 72)
    near(lib.tdg_expert_layer(*(t.cuda() for t in small), workspace=work[1]), *layer64(*small, F16))
    assert torch.equal(lib.tdg_expert_layer(*dev[2], workspace=work[1]), want[2])


def test_wrong_shapes_are_refused(lib):
    p = [t.cuda() for t in problem(rng(1), 4, 2, 3, 16, 8)]
    x, ids, w, up, down = p
    assert lib.tdg_expert_layer(*p).shape == (4, 16)
    for args in ((x[:3], ids, w, up, down), (x, ids, w[:, :1], up, down), (x, ids, w, up[:, :, :15], down),
                 (x, ids, w, up[:2], down), (x, ids, w, up, down[:, :7]), (x, ids, w, up, down[..., :15]),
                 (x, ids, w, up.cpu(), down), (x.t(), ids, w, up, down)):
        with pytest.raises(ValueError):
            lib.tdg_expert_layer(*args)
    with pytest.raises(ValueError):
        lib.tdg_expert_layer(*p, out=torch.zeros(4, 15, device="cuda"))
    with pytest.raises(TypeError):
        lib.tdg_expert_layer(x, ids.long(), w, up, down)
    with pytest.raises(TypeError):
        lib.tdg_expert_layer(x, ids, w.half(), up, down)
    with pytest.raises(lib.TdgError):
        lib.tdg_expert_layer(*p, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    many = torch.zeros(65, 16, dtype=F16, device="cuda")
    with pytest.raises(lib.TdgError):
        lib.tdg_expert_layer(many, torch.zeros(65, 2, dtype=torch.int32, device="cuda"), None, up, down)
