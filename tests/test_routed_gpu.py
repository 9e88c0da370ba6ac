"""GPU tests of the operators whose rows pick their weights, against plain
implementations in 64 bits on the CPU.

Tolerances, from the arithmetic alone (u = 2^-24, half a step of FP32):
  * a sum of n products in FP32, in any order, is off by at most about
    n * 2u * sum |a b| (one rounding per step; twice that, since a matrix
    instruction may truncate inside its sum);
  * rounding to FP16 once adds 2^-11 |y| (and half its smallest step, 2^-25).
Integers small enough that every sum stays below 2^24 have to be exact."""
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


def normal(r, *shape, dtype=F16, scale=1.0):
    return torch.from_numpy(r.standard_normal(shape) * scale).to(dtype)


def whole(r, *shape, most=3, dtype=F16):
    return torch.from_numpy(r.integers(-most, most + 1, shape)).to(dtype)


def wider(t, pad, skip=0):
    """t's values on the device in rows `pad` elements longer, `skip` elements
    into the buffer; what lies between is NaN."""
    buf = torch.full((t.shape[0] * (t.shape[1] + pad) + skip,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[skip:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    v.copy_(t)
    return v


def at_page_end(t):
    """t (a matrix, or a stack) on the device, its last byte the last of a
    4 KiB page; NaN behind it."""
    bytes_ = t.numel() * t.element_size()
    buf = torch.full(((bytes_ + 8192) // t.element_size(),), float("nan"), dtype=t.dtype, device="cuda")
    skip = (-(buf.data_ptr() + bytes_)) % 4096 // t.element_size()
    v = buf[skip:skip + t.numel()].view(t.shape)
    assert (v.data_ptr() + bytes_) % 4096 == 0
    return v.copy_(t)


def near(got, want, tol):
    got = got.cpu().double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%d of %d off, the first at %s: got %r, want %r within %r" % (
        int(bad.sum()), bad.numel(), tuple(bad.nonzero()[0].tolist()), float(got[bad][0]), float(want[bad][0]),
        float(tol[bad][0]))


def out_step(want, dtype):
    return want.abs() * 2.0 ** -11 + 2.0 ** -25 if dtype == F16 else want.abs() * 2.0 ** -24 + 2.0 ** -150


# ------------------------------------------------------------------ the plan

def plan_of(ids, experts):
    flat = ids.reshape(-1)
    of = [np.flatnonzero(flat == e) for e in range(experts)]
    offsets = np.concatenate(([0], np.cumsum([len(o) for o in of])))
    kept = np.concatenate(of)
    order = np.full(flat.size, -1)
    order[:kept.size] = kept
    slots = np.full(flat.size, -1)
    slots[kept] = np.arange(kept.size)
    return offsets, order, slots.reshape(ids.shape)


PLANS = [(1, 1, 1), (1, 8, 128), (5, 8, 7), (63, 1, 2), (64, 1, 64), (65, 3, 1000), (256, 1, 3), (257, 1, 513),
         (4096, 1, 1024), (4097, 1, 1024), (1000, 8, 64), (3001, 7, 255), (20000, 8, 256), (200000, 8, 17)]


@pytest.mark.parametrize("tokens,top_k,experts", PLANS)
@pytest.mark.parametrize("kind", ["mixed", "one", "dropped"])
def test_plan(lib, tokens, top_k, experts, kind):
    r = rng(tokens, top_k, experts)
    ids = r.integers(-2, experts + 2, (tokens, top_k))  # some outside on both sides, repeats
    if kind == "one":
        ids[:] = experts - 1
    elif kind == "dropped":
        ids[:] = -1
        ids.reshape(-1)[::3] = 2 ** 31 - 1
    t = torch.from_numpy(ids).to(torch.int32).cuda()
    got = lib.tdg_route_plan(t, experts)
    for g, w in zip(got, plan_of(ids, experts)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_plan_of_no_tokens(lib):
    offsets, order, slots = lib.tdg_route_plan(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert offsets.tolist() == [0] * 10 and order.numel() == 0 and slots.shape == (0, 4)


def test_plan_of_strided_ids_into_given_outputs(lib):
    ids = rng(5).integers(0, 40, (700, 6))
    wide = torch.full((700, 11), 3, dtype=torch.int32, device="cuda")
    wide[:, 2:8] = torch.from_numpy(ids).to(torch.int32)
    off = torch.full((41,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((4200,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((700, 6), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((lib.tdg_route_workspace(700, 6, 40),), 0xAB, dtype=torch.uint8, device="cuda")
    lib.tdg_route_plan(wide[:, 2:8], 40, off, order, slots, ws)
    for g, w in zip((off, order, slots), plan_of(ids, 40)):
        assert np.array_equal(g.cpu().numpy(), w)


# ------------------------------------------------------------------ rows

ROWS = [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (17, 3, 64), (33, 1, 129), (100, 8, 1000), (9, 5, 4095), (260, 2, 12),
        (2, 9, 20001), (64, 17, 96)]


def routed(r, tokens, top_k, drop=0.2):
    """slots of a plan over 6 experts, some entries (and the last token) dropped."""
    ids = r.integers(0, 6, (tokens, top_k))
    ids[r.random((tokens, top_k)) < drop] = -1
    if tokens > 1:
        ids[-1] = -1
    return torch.from_numpy(plan_of(ids, 6)[2]).to(torch.int32)


def combine64(z, slots, w):
    y = torch.zeros(slots.shape[0], z.shape[1], dtype=torch.float64)
    mag = y.clone()
    for j in range(slots.shape[1]):
        on = (slots[:, j] >= 0).nonzero().reshape(-1)
        rows = z[slots[on, j].long()].double()
        wj = w[on, j].double()[:, None] if w is not None else 1.0
        y[on] += wj * rows
        mag[on] += (wj * rows).abs()
    return y, mag


@pytest.mark.parametrize("tokens,top_k,cols", ROWS)
@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("pad,skip", [(0, 0), (5, 3)])
def test_dispatch(lib, tokens, top_k, cols, dtype, pad, skip):
    r = rng(1, tokens, top_k, cols)
    x, slots = normal(r, tokens, cols, dtype=dtype), routed(r, tokens, top_k)
    x.view(-1)[::7] = float("nan")
    bits = torch.int16 if dtype == F16 else torch.int32
    out = wider(torch.full((tokens * top_k, cols), -7.0, dtype=dtype), pad, skip)
    lib.tdg_rows_dispatch(wider(x, pad, skip), slots.cuda(), out)
    want = torch.full((tokens * top_k, cols), -7.0, dtype=dtype)  # rows without a slot stay
    on = slots >= 0
    want[slots[on].long()] = x[:, None, :].expand(-1, top_k, -1)[on]
    assert torch.equal(out.cpu().contiguous().view(bits), want.view(bits))
    base = out._base.cpu()[skip:].view(tokens * top_k, cols + pad)[:, cols:]
    assert torch.isnan(base).all()  # the gaps between rows too


@pytest.mark.parametrize("tokens,top_k,cols", ROWS)
@pytest.mark.parametrize("rows_t,tok_t", [(F16, F16), (F16, F32), (F32, F16), (F32, F32)])
@pytest.mark.parametrize("weighted,pad,skip", [(True, 0, 0), (True, 3, 1), (False, 0, 0)])
def test_combine(lib, tokens, top_k, cols, rows_t, tok_t, weighted, pad, skip):
    r = rng(2, tokens, top_k, cols)
    z, slots = normal(r, tokens * top_k, cols, dtype=rows_t), routed(r, tokens, top_k)
    w = normal(r, tokens, top_k, dtype=F32) if weighted else None
    used = torch.zeros(z.shape[0], dtype=torch.bool)
    used[slots[slots >= 0].long()] = True
    want, mag = combine64(z, slots, w)
    z[~used] = float("nan")  # rows of no token, weights of no row: never seen
    if weighted:
        w[slots < 0] = float("inf")
    out = wider(torch.zeros(tokens, cols, dtype=tok_t), pad, skip)
    got = lib.tdg_rows_combine(wider(z, pad, skip), slots.cuda(),
                               wider(w, pad) if weighted else None, out)
    assert got is out
    near(got, want, top_k * U2 * mag + out_step(want, tok_t))
    fresh = lib.tdg_rows_combine(z.cuda(), slots.cuda(), w.cuda() if weighted else None, out_dtype=tok_t)
    assert torch.equal(fresh, got)


@pytest.mark.parametrize("tokens,top_k,cols", ROWS)
@pytest.mark.parametrize("rows_t,tok_t", [(F16, F16), (F16, F32), (F32, F16), (F32, F32)])
@pytest.mark.parametrize("weighted,pad,skip", [(True, 0, 0), (True, 3, 1), (False, 0, 0)])
def test_combine_grad(lib, tokens, top_k, cols, rows_t, tok_t, weighted, pad, skip):
    r = rng(3, tokens, top_k, cols)
    z, slots = normal(r, tokens * top_k, cols, dtype=rows_t), routed(r, tokens, top_k)
    dy = normal(r, tokens, cols, dtype=tok_t)
    w = normal(r, tokens, top_k, dtype=F32) if weighted else None
    on = slots >= 0
    at = slots[on].long()
    g = dy.double()[:, None, :].expand(-1, top_k, -1)[on]
    want_z = torch.full((tokens * top_k, cols), -7.0, dtype=torch.float64)
    want_z[at] = (w[on].double()[:, None] if weighted else 1.0) * g
    want_w, mag = torch.zeros(tokens, top_k, dtype=torch.float64), torch.zeros(tokens, top_k, dtype=torch.float64)
    want_w[on] = (g * z[at].double()).sum(dim=1)
    mag[on] = (g * z[at].double()).abs().sum(dim=1)
    unused = torch.ones(z.shape[0], dtype=torch.bool)
    unused[at] = False
    z[unused] = float("nan")
    dz = wider(torch.full((tokens * top_k, cols), -7.0, dtype=rows_t), pad, skip)
    dw = wider(torch.full((tokens, top_k), -7.0), pad)
    got = lib.tdg_rows_combine_grad(wider(dy, pad, skip), wider(z, pad, skip), slots.cuda(),
                                    wider(w, pad) if weighted else None, dz, dw)
    assert got[0] is dz and got[1] is dw
    near(dz, want_z, out_step(want_z, rows_t) * (1 + 2.0 ** -10))  # the FP32 product, then the row's type
    near(dw, want_w, cols * U2 * mag)


def test_slots_beyond_the_rows_have_no_row(lib):
    """A buffer with fewer rows than kept entries, and slots that make no sense."""
    x = torch.arange(12, dtype=F32).reshape(4, 3).cuda() + 1
    slots = torch.tensor([[0, 5], [2, 2 ** 31 - 1], [-2 ** 31, 1], [3, -1]], dtype=torch.int32).cuda()
    out = torch.zeros(3, 3, device="cuda")
    lib.tdg_rows_dispatch(x, slots, out)
    assert torch.equal(out, x[[0, 2, 1]])
    y = lib.tdg_rows_combine(out, slots)
    assert torch.equal(y.cpu(), torch.cat((x[:3].cpu(), torch.zeros(1, 3))))
    dz, dw = lib.tdg_rows_combine_grad(x, out, slots)
    assert torch.equal(dz, out)
    assert torch.equal(dw.cpu() != 0, torch.tensor([[True, False], [True, False], [False, True], [False, False]]))


def test_row_gradients_against_differences(lib):
    """combine is linear in z and in w: whole differences give its gradient."""
    r = rng(4)
    T, k, H = 13, 3, 70
    slots = routed(r, T, k).cuda()
    z, w, dy = (whole(r, *s, dtype=F32).cuda() for s in ((T * k, H), (T, k), (T, H)))
    dz, dw = lib.tdg_rows_combine_grad(dy, z, slots, w, dz=torch.zeros_like(z))
    value = lambda z, w: float((lib.tdg_rows_combine(z, slots, w) * dy).double().sum())
    base = value(z, w)
    for i, j in ((0, 0), (5, 2), (12, 1), (7, 0)):
        step = w.clone()
        step[i, j] += 1
        assert value(z, step) - base == float(dw[i, j])
        step = z.clone()
        step[i * k + j, 11 * j] += 1
        assert value(step, w) - base == float(dz[i * k + j, 11 * j])
    # dispatch's gradient is the combine without weights
    x, dout = whole(r, T, H, dtype=F32).cuda(), whole(r, T * k, H, dtype=F32).cuda()
    out = lib.tdg_rows_dispatch(x, slots, torch.zeros(T * k, H, device="cuda"))
    dx = lib.tdg_rows_combine(dout, slots)
    assert float((out * dout).double().sum()) == float((x * dx).double().sum())


def test_rows_past_32_bits(lib):
    """Sorted rows whose byte offsets pass 2^32, and whose elements pass 2^31."""
    rows, cols = 550000, 4096
    z = torch.zeros(rows, cols, dtype=F16, device="cuda")
    x = normal(rng(6), 2, cols).cuda()
    slots = torch.tensor([[rows - 1, 3], [rows - 2, 530001]], dtype=torch.int32, device="cuda")
    lib.tdg_rows_dispatch(x, slots, z)
    assert torch.equal(z[[rows - 1, 3, rows - 2, 530001]], x[[0, 0, 1, 1]])
    assert int((z != 0).any(dim=1).sum()) == 4
    assert torch.equal(lib.tdg_rows_combine(z, slots), 2 * x)


# ------------------------------------------------------------------ the experts' products

GROUPED = [  # rows of each group, K, N
    ([1], 1, 1), ([0], 8, 8), ([3, 0, 5], 16, 24), ([0, 0, 130, 0], 64, 64), ([1] * 40, 72, 40),
    ([127, 128, 129], 128, 136), ([300, 1, 0, 257], 200, 264), ([31, 32, 33, 64, 65], 65, 67),
    ([5, 70], 1000, 33), ([7, 2, 9], 7, 300), ([40] * 70, 40, 16), ([600], 520, 512), ([260, 20, 500], 264, 250),
    ([2, 30, 1, 4], 2048, 96), ([64, 64], 0, 16), ([513, 255], 96, 320),
    # enough tiles for the larger ones, and for several of them per workgroup
    ([300, 200], 72, 6400), ([300, 200], 72, 9001), ([1100, 947], 72, 8200), ([20, 31], 1000, 1600),
    ([20, 31], 1000, 2400), ([3, 0, 70, 1] * 66, 264, 250),
    # many groups of a few rows
    ([2, 0, 1, 5] * 11 + [60], 200, 1000), ([1, 3] * 15 + [33, 32], 65, 777), ([4, 1] * 13, 520, 1030),
    # several rounds of the largest tiles
    ([2000, 1990], 200, 4100), ([1990, 2055], 321, 4097), ([3, 0, 70, 1] * 16 + [5, 2], 510, 1023),
    ([64, 1, 0, 130] * 16, 512, 1024),
]


def groups_of(rows, before=2, behind=3):
    """offsets (with rows of no group at both ends) and the row count."""
    off = np.cumsum([before] + rows)
    return torch.from_numpy(off).to(torch.int32), int(off[-1]) + behind


def grouped64(a, b, off):
    y, mag = (torch.full((a.shape[0], b.shape[2]), -7.0, dtype=torch.float64) for _ in range(2))
    for g in range(b.shape[0]):
        s = slice(int(off[g]), int(off[g + 1]))
        y[s] = a[s].double() @ b[g].double()
        mag[s] = a[s].double().abs() @ b[g].double().abs()
    return y, mag


def stacked(t, pad, skip, gap):
    """A stack in wider rows, `gap` elements between matrices; NaN in between."""
    n, r, c = t.shape
    size = r * (c + pad) + gap
    buf = torch.full((n * size + skip,), float("nan"), dtype=t.dtype, device="cuda")
    v = torch.as_strided(buf, (n, r, c), (size, c + pad, 1), skip)
    v.copy_(t)
    return v


LAYOUTS = [(0, 0, 0), (8, 8, 16), (3, 1, 5)]


@pytest.mark.parametrize("rows,K,N", GROUPED)
@pytest.mark.parametrize("pad,skip,gap", LAYOUTS)
@pytest.mark.parametrize("kind", ["whole", "normal"])
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped(lib, rows, K, N, pad, skip, gap, kind, transposed):
    r = rng(7, len(rows), K, N)
    off, R = groups_of(rows)
    make = whole if kind == "whole" else normal
    a, b = make(r, R, K), make(r, len(rows), K, N)
    want, mag = grouped64(a, b, off)
    inside = torch.zeros(R, dtype=torch.bool)
    inside[int(off[0]):int(off[-1])] = True
    a[~inside] = float("nan")
    bt = b.transpose(1, 2).contiguous() if transposed else b
    C = wider(torch.full((R, N), -7.0), pad, skip)
    fn = lib.gemm_f16f32_grouped_nt if transposed else lib.gemm_f16f32_grouped
    got = fn(wider(a, pad, skip), stacked(bt, pad, skip, gap), off.cuda(), C)
    tol = torch.zeros_like(want) if kind == "whole" else K * U2 * mag.clamp(min=0)
    tol[~inside] = 0
    near(got, want, tol)


@pytest.mark.parametrize("rows,M,N", GROUPED)
@pytest.mark.parametrize("pad,skip,gap", LAYOUTS)
@pytest.mark.parametrize("kind", ["whole", "normal"])
def test_grouped_tn(lib, rows, M, N, pad, skip, gap, kind):
    r = rng(8, len(rows), M, N)
    off, R = groups_of(rows)
    make = whole if kind == "whole" else normal
    a, b = make(r, R, M), make(r, R, N)
    G = len(rows)
    want, tol = torch.zeros(G, M, N, dtype=torch.float64), torch.zeros(G, M, N, dtype=torch.float64)
    for g in range(G):
        s = slice(int(off[g]), int(off[g + 1]))
        want[g] = a[s].double().t() @ b[s].double()
        if kind == "normal":
            tol[g] = rows[g] * U2 * (a[s].double().abs().t() @ b[s].double().abs())
    for t in (a, b):
        t[:int(off[0])] = float("nan")
        t[int(off[-1]):] = float("nan")
    C = stacked(torch.full((G, M, N), -7.0), pad, skip, gap)
    got = lib.gemm_f16f32_grouped_tn(wider(a, pad, skip), wider(b, pad, skip), off.cuda(), C)
    near(got, want, tol)


@pytest.mark.parametrize("rows,K,N", [([40, 0, 70], 65, 67), ([1], 1, 1), ([300, 20], 96, 129), ([5], 129, 96),
                                      ([2, 260], 1001, 7)])
def test_grouped_operands_at_a_page_end(lib, rows, K, N):
    """Operands with nothing mapped to count on behind them."""
    r = rng(20, K, N)
    off, R = groups_of(rows, 0, 0)
    a, b, dy = whole(r, R, K), whole(r, len(rows), K, N), whole(r, R, N)
    o, zero = off.cuda(), lambda t: torch.zeros_like(t)
    want, _ = grouped64(a, b, off)
    near(lib.gemm_f16f32_grouped(at_page_end(a), at_page_end(b), o), want, zero(want))
    bt = b.transpose(1, 2).contiguous()
    near(lib.gemm_f16f32_grouped_nt(at_page_end(a), at_page_end(bt), o), want, zero(want))
    want = torch.stack([a[int(off[g]):int(off[g + 1])].double().t() @ dy[int(off[g]):int(off[g + 1])].double()
                        for g in range(len(rows))])
    near(lib.gemm_f16f32_grouped_tn(at_page_end(a), at_page_end(dy), o), want, zero(want))


@pytest.mark.parametrize("M,K,N,rank", [(3, 65, 67, 9), (70, 129, 130, 33), (300, 97, 255, 5)])
def test_lora_operands_at_a_page_end(lib, M, K, N, rank):
    r = rng(21, M)
    a, b, down, up = whole(r, M, K, most=2), whole(r, K, N), whole(r, 3, K, rank, most=1), whole(r, 3, rank, N, most=2)
    pick = torch.from_numpy(r.integers(-1, 3, M)).to(torch.int32)
    want, _, _ = lora64(a, b, down, up, pick, None)
    got = lib.gemm_f16f32_lora(at_page_end(a), at_page_end(b), at_page_end(down), at_page_end(up), pick.cuda())
    near(got, want, torch.zeros_like(want))


def wide_at_page_end(t, pad):
    """As at_page_end, rows of `pad` elements more (the last one without)."""
    n, r, c = t.shape if t.dim() == 3 else (1,) + tuple(t.shape)
    flat = torch.full((n * r, c + pad), float("nan"), dtype=t.dtype)
    flat[:, :c] = t.reshape(n * r, c)
    held = at_page_end(flat.reshape(-1)[:(n * r - 1) * (c + pad) + c])
    v = torch.as_strided(held, (n, r, c), (r * (c + pad), c + pad, 1))
    return v if t.dim() == 3 else v[0]


# each of the tiles, k in one, two and more steps, whole and cut, a few columns
PAGE_ENDS = [([40, 0, 70], 64, 67), ([64, 128], 128, 129), ([128, 64], 192, 131), ([9, 64], 320, 65),
             ([100, 28], 128, 3), ([70], 64, 1), ([33, 30], 65, 7), ([64], 8, 9), ([300, 212], 64, 9001),
             ([300, 200], 72, 6403), ([1100, 948], 71, 8201), ([20, 31], 1000, 1601), ([64, 192], 256, 2401),
             ([3, 0, 70, 1] * 66, 263, 251), ([1, 3] * 15 + [33, 31], 64, 777), ([4, 1] * 13, 521, 1029),
             ([2, 0, 5] * 20, 192, 1001), ([2000, 1990], 321, 4099), ([3, 0, 64, 1] * 16 + [5, 2], 511, 1023)]


@pytest.mark.parametrize("rows,K,N", PAGE_ENDS)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_grouped_tiles_at_a_page_end(lib, rows, K, N, pad):
    r = rng(29, K, N, pad)
    off, R = groups_of(rows, 0, 0)
    a, b, dy = whole(r, R, K), whole(r, len(rows), K, N), whole(r, R, N)
    o, zero, end = off.cuda(), lambda t: torch.zeros_like(t), lambda t: wide_at_page_end(t, pad)
    want, _ = grouped64(a, b, off)
    near(lib.gemm_f16f32_grouped(end(a), end(b), o), want, zero(want))
    near(lib.gemm_f16f32_grouped(a.cuda(), end(b), o), want, zero(want))
    near(lib.gemm_f16f32_grouped(end(a), b.cuda(), o), want, zero(want))
    bt = b.transpose(1, 2).contiguous()
    near(lib.gemm_f16f32_grouped_nt(end(a), end(bt), o), want, zero(want))
    near(lib.gemm_f16f32_grouped_nt(a.cuda(), end(bt), o), want, zero(want))
    want = torch.stack([a[int(off[g]):int(off[g + 1])].double().t() @ dy[int(off[g]):int(off[g + 1])].double()
                        for g in range(len(rows))])
    near(lib.gemm_f16f32_grouped_tn(end(a), end(dy), o), want, zero(want))
    near(lib.gemm_f16f32_grouped_tn(a.cuda(), end(dy), o), want, zero(want))


@pytest.mark.parametrize("M,K,N,rank", [(3, 64, 67, 8), (20, 128, 129, 9), (70, 192, 131, 33), (256, 65, 7, 3),
                                        (300, 64, 129, 16), (257, 128, 3, 1), (400, 72, 1001, 40), (600, 130, 5001, 9),
                                        (1100, 64, 6601, 17), (1100, 71, 6603, 65), (700, 64, 2305, 17),
                                        (700, 71, 2303, 65)])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_lora_tiles_at_a_page_end(lib, M, K, N, rank, pad):
    r = rng(30, M, K, pad)
    a, b, down, up = whole(r, M, K, most=2), whole(r, K, N), whole(r, 3, K, rank, most=1), whole(r, 3, rank, N, most=2)
    pick = torch.from_numpy(r.integers(-1, 3, M)).to(torch.int32)
    want, _, _ = lora64(a, b, down, up, pick, None)
    plain = [t.cuda() for t in (a, b, down, up)]
    ends = [wide_at_page_end(t, pad) for t in (a, b, down, up)]
    for args in (ends, [ends[0]] + plain[1:], plain[:1] + [ends[1]] + plain[2:], plain[:2] + [ends[2], plain[3]],
                 plain[:3] + [ends[3]]):
        near(lib.gemm_f16f32_lora(*args, pick.cuda()), want, torch.zeros_like(want))


def apart_at_page_ends(t, pad):
    """A stack whose matrices each end with a page, with a page of NaN or more
    before the next one; rows of `pad` elements more."""
    n, r, c = t.shape
    span = (r - 1) * (c + pad) + c
    stride = (span + 2047) // 2048 * 2048 + 2048
    buf = torch.full((n * stride + 4096,), float("nan"), dtype=t.dtype, device="cuda")
    skip = (-(buf.data_ptr() + span * 2)) % 4096 // 2
    v = torch.as_strided(buf, (n, r, c), (stride, c + pad, 1), skip)
    assert all((v[g].data_ptr() + span * 2) % 4096 == 0 for g in range(n))
    return v.copy_(t)


@pytest.mark.parametrize("rows,K,N", PAGE_ENDS)
@pytest.mark.parametrize("pad", [0, 3])
def test_grouped_weights_apart_at_page_ends(lib, rows, K, N, pad):
    r = rng(34, K, N, pad)
    off, R = groups_of(rows, 0, 0)
    a, b = whole(r, R, K), whole(r, len(rows), K, N)
    want, _ = grouped64(a, b, off)
    near(lib.gemm_f16f32_grouped(a.cuda(), apart_at_page_ends(b, pad), off.cuda()), want, torch.zeros_like(want))
    bt = b.transpose(1, 2).contiguous()
    near(lib.gemm_f16f32_grouped_nt(a.cuda(), apart_at_page_ends(bt, pad), off.cuda()), want, torch.zeros_like(want))


@pytest.mark.parametrize("M,K,N,rank", [(3, 64, 67, 8), (20, 128, 129, 9), (70, 192, 131, 33), (256, 65, 7, 3),
                                        (300, 64, 129, 17), (400, 72, 1001, 41), (1100, 71, 6603, 65),
                                        (700, 64, 2305, 17), (700, 71, 2303, 5)])
@pytest.mark.parametrize("pad", [0, 3])
def test_lora_adapters_apart_at_page_ends(lib, M, K, N, rank, pad):
    r = rng(35, M, K, pad)
    a, b, down, up = whole(r, M, K, most=2), whole(r, K, N), whole(r, 3, K, rank, most=1), whole(r, 3, rank, N, most=2)
    pick = torch.from_numpy(r.integers(-1, 3, M)).to(torch.int32)
    want, _, _ = lora64(a, b, down, up, pick, None)
    got = lib.gemm_f16f32_lora(a.cuda(), b.cuda(), apart_at_page_ends(down, pad), apart_at_page_ends(up, pad), pick.cuda())
    near(got, want, torch.zeros_like(want))


@pytest.mark.parametrize("K,N", [(128, 128), (72, 100), (65, 67)])
def test_groups_do_not_touch_each_other(lib, K, N):
    """Infinities and NaN in one group's rows and weights stay in that group."""
    r = rng(9)
    rows = [70, 40, 90]
    off, R = groups_of(rows, 0, 0)
    a, b, dy = whole(r, R, K), whole(r, 3, K, N), whole(r, R, N)
    sick = slice(70, 110)
    well = torch.ones(R, dtype=torch.bool)
    well[sick] = False
    clean = [x.cpu() for x in (lib.gemm_f16f32_grouped(a.cuda(), b.cuda(), off.cuda()),
                               lib.gemm_f16f32_grouped_nt(dy.cuda(), b.cuda(), off.cuda()),
                               lib.gemm_f16f32_grouped_tn(a.cuda(), dy.cuda(), off.cuda()))]
    a[sick], b[1], dy[sick] = float("inf"), float("nan"), float("nan")
    y = lib.gemm_f16f32_grouped(a.cuda(), b.cuda(), off.cuda()).cpu()
    dx = lib.gemm_f16f32_grouped_nt(dy.cuda(), b.cuda(), off.cuda()).cpu()
    dw = lib.gemm_f16f32_grouped_tn(a.cuda(), dy.cuda(), off.cuda()).cpu()
    assert torch.equal(y[well], clean[0][well]) and torch.isnan(y[sick]).all()
    assert torch.equal(dx[well], clean[1][well]) and torch.isnan(dx[sick]).all()
    assert torch.equal(dw[[0, 2]], clean[2][[0, 2]]) and torch.isnan(dw[1]).all()


def test_grouped_gradients_against_differences(lib):
    """The product is linear in each operand: whole differences are exact."""
    r = rng(10)
    off, R = groups_of([50, 0, 131, 9], 0, 0)
    K, N = 72, 88
    o = off.cuda()
    a, b, dy, da, db = (whole(r, *s).cuda() for s in ((R, K), (4, K, N), (R, N), (R, K), (4, K, N)))
    dot = lambda x, y: float((x.double() * y.double()).sum())
    y = lib.gemm_f16f32_grouped(a, b, o)
    dx, dw = lib.gemm_f16f32_grouped_nt(dy, b, o), lib.gemm_f16f32_grouped_tn(a, dy, o)
    assert dot(lib.gemm_f16f32_grouped(a + da, b, o) - y, dy) == dot(dx, da)
    assert dot(lib.gemm_f16f32_grouped(a, b + db, o) - y, dy) == dot(dw, db)


def test_one_weight_for_all_groups_and_many_groups(lib):
    r = rng(11)
    rows = list(r.integers(0, 4, 1024))
    off, R = groups_of(rows, 0, 0)
    a, b = whole(r, R, 40), whole(r, 1, 40, 24)
    got = lib.gemm_f16f32_grouped(a.cuda(), b.cuda().expand(1024, -1, -1), off.cuda())
    near(got, a.double() @ b[0].double(), torch.zeros(R, 24, dtype=torch.float64))


@pytest.mark.parametrize("offsets", [[-5, 40, 30, 1000, 2 ** 31 - 1], [60, 50, 40, 30, 20], [-2 ** 31] * 5,
                                     [0, 1000, 0, 1000, 0]])
def test_offsets_that_make_no_sense_stay_inside(lib, offsets):
    """Nothing is read or written outside the arrays, whatever the offsets say."""
    a, b = torch.ones(64, 32, dtype=F16, device="cuda"), torch.ones(4, 32, 48, dtype=F16, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    buf = torch.full((80, 48), -7.0, device="cuda")
    lib.gemm_f16f32_grouped(a, b, off, buf[8:72])
    assert bool((buf[:8] == -7).all()) and bool((buf[72:] == -7).all())
    assert bool(((buf == -7) | (buf == 32)).all())
    dw = lib.gemm_f16f32_grouped_tn(a, a, off)
    assert bool(torch.isfinite(dw).all()) and float(dw.max()) <= 64


def wild_offsets(r, kind, groups, R):
    if kind == "descending":
        off = np.sort(r.integers(0, R + 1, groups + 1))[::-1]
    elif kind == "around":
        off = r.integers(-R, 2 * R + 1, groups + 1)
    elif kind == "anywhere":
        off = r.integers(-2 ** 31, 2 ** 31, groups + 1)
    else:  # the whole range again and again
        off = np.where(np.arange(groups + 1) % 2 == 0, -2 ** 31, 2 ** 31 - 1)
    return torch.from_numpy(off.copy()).to(torch.int32)


@pytest.mark.parametrize("rows,K,N", GROUPED[2:3] + GROUPED[6:8] + GROUPED[16:] + [([2, 260], 1001, 7)])
@pytest.mark.parametrize("kind", ["descending", "around", "anywhere", "all"])
def test_wild_offsets_in_every_tile(lib, rows, K, N, kind):
    """Offsets that do not ascend or lie outside the rows, for each of the tiles
    (the last shape's weights end with a page: the register path).  They count
    as clamped to the rows.  A row of several groups has the product of one of
    them, or none where there are more tiles than the rows can make; a row of
    no group stays as it was, and so does all around C."""
    r = rng(36, K, N, len(rows))
    G, R = len(rows), sum(rows)
    a, b, dy = whole(r, R, K, most=1), whole(r, G, K, N, most=1), whole(r, R, N, most=1)
    off = wild_offsets(r, kind, G, R)
    at = off.long().clamp(0, R).tolist()
    end = at_page_end if N == 7 else (lambda t: t.cuda())
    for fn, w in ((lib.gemm_f16f32_grouped, b), (lib.gemm_f16f32_grouped_nt, b.transpose(1, 2).contiguous())):
        buf = torch.full((R + 16, N), -7.5, device="cuda")
        fn(a.cuda(), end(w), off.cuda(), buf[8:R + 8])
        got = buf.cpu()
        assert (got[:8] == -7.5).all() and (got[R + 8:] == -7.5).all()
        got = got[8:R + 8]
        fine = got == -7.5
        for g in range(G):
            if at[g + 1] > at[g]:
                s = slice(at[g], at[g + 1])
                fine[s] |= got[s] == a[s].float() @ b[g].float()
        assert fine.all()
        ascending = [g for g in range(G) if at[g + 1] > at[g]]
        if len(ascending) == 1:  # and then every row of it has its product
            s = slice(at[ascending[0]], at[ascending[0] + 1])
            assert not (got[s] == -7.5).any()
    buf = torch.full((G + 2, K, N), -7.5, device="cuda")
    lib.gemm_f16f32_grouped_tn(a.cuda(), end(dy), off.cuda(), buf[1:G + 1])
    got = buf.cpu()
    assert (got[0] == -7.5).all() and (got[G + 1] == -7.5).all()
    for g in range(G):
        s = slice(at[g], max(at[g], at[g + 1]))
        assert torch.equal(got[g + 1], a[s].float().t() @ dy[s].float())


def test_grouped_past_32_bits(lib):
    """Weights and rows whose byte offsets pass 2^32."""
    r = rng(12)
    G, K, N = 3, 32768, 32768
    b = torch.zeros(G, K, N, dtype=F16, device="cuda")
    small = whole(r, G, 64, N).cuda()
    b[:, K - 64:] = small
    a = whole(r, 6, K)
    off = torch.tensor([0, 1, 3, 6], dtype=torch.int32, device="cuda")
    got = lib.gemm_f16f32_grouped(a.cuda(), b, off).cpu()
    for g, s in enumerate((slice(0, 1), slice(1, 3), slice(3, 6))):
        assert torch.equal(got[s].double(), a[s, K - 64:].double() @ small[g].cpu().double())


@pytest.mark.parametrize("far", [8388351, 8388352, 8388353, 9000000])
def test_grouped_rows_far_apart(lib, far):
    """Leading dimensions around and past what a lane's 32-bit offsets reach,
    each operand in turn; and rows that all lie in one group."""
    r = rng(23)
    off = torch.tensor([0, 30, 260], dtype=torch.int32, device="cuda")
    a, b, dy = whole(r, 260, 40), whole(r, 2, 40, 24), whole(r, 260, 24)
    want, _ = grouped64(a, b, off.cpu())
    buf = torch.zeros(259 * far + 64, dtype=F16, device="cuda")
    wide = lambda t: torch.as_strided(buf, tuple(t.shape), (far, 1), 5).copy_(t)
    deep = lambda t: torch.as_strided(buf, tuple(t.shape), (t.shape[1] * far, far, 1), 3).copy_(t)
    same = lambda got, want: near(got, want, torch.zeros_like(want))
    same(lib.gemm_f16f32_grouped(wide(a), b.cuda(), off), want)
    same(lib.gemm_f16f32_grouped(a.cuda(), deep(b), off), want)
    bt = b.transpose(1, 2).contiguous()
    same(lib.gemm_f16f32_grouped_nt(a.cuda(), deep(bt), off), want)
    dw = torch.stack([a[:30].double().t() @ dy[:30].double(), a[30:].double().t() @ dy[30:].double()])
    same(lib.gemm_f16f32_grouped_tn(wide(a), dy.cuda(), off), dw)
    same(lib.gemm_f16f32_grouped_tn(a.cuda(), wide(dy), off), dw)


@pytest.mark.parametrize("far", [8388352, 8388353])
def test_grouped_large_tiles_far_apart(lib, far):
    """The same for 256 rows by 256 columns at a time."""
    r = rng(26)
    off = torch.tensor([0, 260], dtype=torch.int32, device="cuda")
    a, b = whole(r, 260, 40), whole(r, 1, 40, 65536)
    buf = torch.zeros(259 * far + 64, dtype=F16, device="cuda")
    a_far = torch.as_strided(buf, (260, 40), (far, 1), 7).copy_(a)
    got = lib.gemm_f16f32_grouped(a_far, b.cuda(), off)
    want = (a.float() @ b[0].float()).double()  # small whole numbers: exact
    near(got, want, torch.zeros_like(want))
    bt = whole(r, 1, 300, 40)
    a2 = whole(r, 60000, 40)
    bt_far = torch.as_strided(buf.zero_()[:259 * far + 64], (1, 260, 40), (260 * far, far, 1), 7).copy_(bt[:, :260])
    off2 = torch.tensor([0, 60000], dtype=torch.int32, device="cuda")
    want = (a2.float() @ bt[0, :260].float().t()).double()
    near(lib.gemm_f16f32_grouped_nt(a2.cuda(), bt_far, off2), want, torch.zeros_like(want))


def test_grouped_without_rows(lib):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 40, dtype=F16, device="cuda")
    dw = lib.gemm_f16f32_grouped_tn(none, torch.empty(0, 24, dtype=F16, device="cuda"), off,
                                    torch.full((3, 40, 24), -7.0, device="cuda"))
    assert not dw.any()
    big = lib.gemm_f16f32_grouped_tn(torch.empty(0, 2048, dtype=F16, device="cuda"),
                                     torch.empty(0, 8192, dtype=F16, device="cuda"), off)
    assert big.shape == (3, 2048, 8192) and not big.any()
    assert lib.gemm_f16f32_grouped(none, torch.ones(3, 40, 24, dtype=F16, device="cuda"), off).shape == (0, 24)


# ------------------------------------------------------------------ adapters

LORA = [  # M, K, N, adapters, rank, tokens of a request
    (1, 1, 1, 1, 1, 1), (1, 4096, 256, 4, 16, 1), (5, 64, 40, 3, 8, 1), (16, 512, 320, 16, 16, 1),
    (33, 100, 67, 5, 9, 4), (64, 1000, 129, 70, 33, 1), (130, 256, 264, 2, 64, 50), (300, 72, 300, 7, 1, 9),
    (257, 520, 512, 6, 128, 40), (40, 48, 64, 4, 256, 3), (513, 128, 136, 3, 16, 300), (700, 65, 35, 9, 17, 1),
    (12, 0, 24, 2, 4, 2), (9, 64, 32, 0, 8, 1), (9, 64, 32, 3, 0, 1),
    # more rows: their product cut in K or not
    (277, 1023, 410, 30, 4, 7), (700, 640, 4100, 5, 20, 40), (4100, 300, 130, 3, 65, 1), (320, 1100, 4090, 9, 33, 3),
]


def lora64(a, b, down, up, pick, scale):
    """The values, the shared part's sum of magnitudes, and the adapters' error bound."""
    M, K = a.shape
    x = a.double()
    y, mag = x @ b.double(), x.abs() @ b.double().abs()
    side = torch.zeros_like(y)
    rank = down.shape[2]
    for i in range(down.shape[0]):
        rows = (pick == i).nonzero().reshape(-1)
        if not rows.numel() or not rank:
            continue
        d, u, s = down[i].double(), up[i].double(), float(scale[i]) if scale is not None else 1.0
        low = x[rows] @ d
        # low itself: a K-long sum, kept to 21 bits; then a rank-long sum
        err = K * U2 * (x[rows].abs() @ d.abs()) + low.abs() * 2.0 ** -21
        y[rows] += s * (low @ u)
        side[rows] = abs(s) * ((err + (rank + 4) * U2 * low.abs()) @ u.abs())
    return y, mag, side


@pytest.mark.parametrize("M,K,N,n,rank,run", LORA)
@pytest.mark.parametrize("pad,skip,gap,scaled", [(0, 0, 0, True), (8, 8, 16, False), (3, 1, 5, True)])
def test_lora(lib, M, K, N, n, rank, run, pad, skip, gap, scaled):
    r = rng(13, M, K, N, n, rank)
    a, b = normal(r, M, K), normal(r, K, N, scale=max(K, 1) ** -0.5)
    down, up = normal(r, n, K, rank, scale=max(K, 1) ** -0.5), normal(r, n, rank, N)
    scale = normal(r, n, dtype=F32) if scaled else None
    pick = torch.from_numpy(np.repeat(r.integers(-1, n + 1, -(-M // run)), run)[:M]).to(torch.int32)
    want, mag, side = lora64(a, b, down, up, pick, scale)
    C = wider(torch.full((M, N), -7.0), pad, skip)
    args = (wider(a, pad, skip), wider(b, pad, skip), stacked(down, pad, skip, gap), stacked(up, pad, skip, gap),
            pick.cuda(), scale.cuda() if scaled else None)
    got = lib.gemm_f16f32_lora(*args, C)
    near(got, want, (K + 2) * U2 * mag + side + want.abs() * 2 * U2)
    ws = torch.full((lib.tdg_lora_workspace(M, N, K, n, rank),), 0xFF, dtype=torch.uint8, device="cuda")
    again = lib.gemm_f16f32_lora(*args, workspace=ws)  # a workspace full of NaN
    assert torch.equal(again, got)


@pytest.mark.parametrize("M,run", [(24, 1), (300, 7), (600, 200)])
@pytest.mark.parametrize("N", [160, 4100])
def test_adapters_do_not_touch_each_other(lib, M, N, run):
    """NaN in one adapter, infinities in another: only their rows see them."""
    r = rng(14, M)
    K, n, rank = 96, 4, 16
    a, b = normal(r, M, K), normal(r, K, N)
    down, up = normal(r, n, K, rank), normal(r, n, rank, N)
    pick = torch.from_numpy(np.repeat(r.integers(-1, n, -(-M // run)), run)[:M]).to(torch.int32)
    dev = lambda: (a.cuda(), b.cuda(), down.cuda(), up.cuda(), pick.cuda())
    clean = lib.gemm_f16f32_lora(*dev()).cpu()
    up[1], down[2] = float("nan"), float("inf")
    got = lib.gemm_f16f32_lora(*dev()).cpu()
    well = (pick != 1) & (pick != 2)
    assert torch.equal(got[well], clean[well])
    assert not torch.isfinite(got[~well]).any()
    plain = lib.gemm_f16f32_pipelined(a.cuda(), b.cuda()).cpu().double()
    none = pick < 0
    tol = K * U2 * (a.double().abs() @ b.double().abs())
    near(got[none], plain[none], 2 * tol[none])


@pytest.mark.parametrize("M,far", [(5, 8388352), (200, 8388352), (255, 8388352), (256, 8388352), (5, 9000000),
                                   (200, 9000000), (600, 9000000), (1000, 2147483), (1000, 2147484)])
@pytest.mark.parametrize("N", [56, 3000])
def test_lora_operands_far_apart(lib, M, N, far):
    """Leading dimensions around and past what a lane's 32-bit offsets reach."""
    r = rng(24, M)
    K, n, rank = 40, 2, 6
    a, b, down, up = whole(r, M, K, most=2), whole(r, K, N), whole(r, n, K, rank, most=1), whole(r, n, rank, N)
    pick = torch.from_numpy(r.integers(-1, n, M)).to(torch.int32)
    want, _, _ = lora64(a, b, down, up, pick, None)
    buf = torch.zeros(max(M, n * K) * far + 64, dtype=F16, device="cuda")
    at = lambda t, i: (torch.as_strided(buf, tuple(t.shape), (far, 1), 3) if t.dim() == 2 else torch.as_strided(
        buf, tuple(t.shape), (t.shape[1] * far, far, 1), 3)).copy_(t)
    for i in range(4):
        args = [t.cuda() for t in (a, b, down, up)]
        args[i] = at((a, b, down, up)[i], i)
        near(lib.gemm_f16f32_lora(*args, pick.cuda()), want, torch.zeros_like(want))


@pytest.mark.parametrize("M", [7, 200, 300])
def test_lora_few_columns(lib, M):
    """Every number of columns around a thread's share of them; the columns
    beside C's stay as they were."""
    r = rng(27, M)
    for N in list(range(1, 10)) + [1021, 1023, 1026, 2049]:
        a, b, down, up = whole(r, M, 40, most=2), whole(r, 40, N), whole(r, 3, 40, 6, most=1), whole(r, 3, 6, N)
        pick = torch.from_numpy(r.integers(-1, 3, M)).to(torch.int32)
        want, _, _ = lora64(a, b, down, up, pick, None)
        buf = torch.full((M, N + 3), -7.0, device="cuda")
        lib.gemm_f16f32_lora(a.cuda(), b.cuda(), down.cuda(), up.cuda(), pick.cuda(), C=buf[:, 1:N + 1])
        near(buf[:, 1:N + 1], want, torch.zeros_like(want))
        assert (buf[:, 0] == -7.0).all() and (buf[:, N + 1:] == -7.0).all()


@pytest.mark.parametrize("N", [72, 200])
def test_lora_many_adapters_and_one_workspace(lib, N):
    """More adapters than the sort has counters, rows over several of its
    blocks, and one workspace for calls of different sizes on one stream."""
    r = rng(25)
    K, n, rank = 48, 3000, 8
    down, up = whole(r, n, K, rank, most=1), whole(r, n, rank, N, most=2)
    b = whole(r, K, N)
    rows = (9000, 300, 100, 4097, 20)
    ws = torch.empty(max(lib.tdg_lora_workspace(M, N, K, n, rank) for M in rows), dtype=torch.uint8, device="cuda")
    for M in rows:
        a = whole(r, M, K, most=2)
        pick = torch.from_numpy(r.integers(-1, n, M)).to(torch.int32)
        x, at = a.double(), pick.clamp(min=0).long()
        low = torch.bmm(x[:, None, :], down.double()[at])
        want = x @ b.double() + torch.bmm(low, up.double()[at])[:, 0] * (pick >= 0)[:, None]
        got = lib.gemm_f16f32_lora(a.cuda(), b.cuda(), down.cuda(), up.cuda(), pick.cuda(), workspace=ws)
        near(got, want, torch.zeros_like(want))


@pytest.mark.parametrize("M,N", [(3, 96), (400, 96), (400, 4000), (1000, 4000), (2200, 3900)])
@pytest.mark.parametrize("size", [2.0 ** -20, 1.0, 2.0 ** 14])
def test_lora_low_products_of_any_size(lib, M, N, size):
    """A . down beyond FP16's range on both sides keeps its bits: rows of very
    different sizes, with whole numbers small enough to be exact."""
    r = rng(15, M)
    K, n, rank = 64, 2, 8
    a = whole(r, M, K, most=2).float()
    a[::2] *= 256.0
    a = a.to(F16)
    b = torch.zeros(K, N, dtype=F16)
    down, up = (whole(r, n, K, rank, most=1).float() * size).to(F16), whole(r, n, rank, N, most=2)
    pick = torch.from_numpy(r.integers(0, n, M)).to(torch.int32)
    want, _, _ = lora64(a, b, down, up, pick, None)
    got = lib.gemm_f16f32_lora(a.cuda(), b.cuda(), down.cuda(), up.cuda(), pick.cuda())
    near(got, want, torch.zeros_like(want))


# few rows; many rows cut in K; and each of the tiles that add low . up
LOW_SHAPES = [(3, 96), (400, 96), (400, 4000), (1000, 4000), (2200, 3900)]


def columns_of_any_size(r, K, n, rank, first, last):
    """down and up of whole numbers, down's columns scaled by powers of two
    from 2^first to 2^last and up's rows so that products are multiples of
    2^-10."""
    size = torch.tensor([2.0 ** round(first + (last - first) * c / (rank - 1)) for c in range(rank)])
    down = whole(r, n, K, rank, most=1).float() * size
    up = whole(r, n, rank, 1, most=1).float() / size[:, None] / 1024
    assert down.abs().max() < 65504 and up.abs().max() < 65504 / 2
    return down.to(F16), up.to(F16)


@pytest.mark.parametrize("M,N", LOW_SHAPES)
@pytest.mark.parametrize("first,last", [(0, -20), (-18, 14), (14, -24)])
def test_lora_elements_of_any_size_in_a_row(lib, M, N, first, last):
    """A . down's elements of one row up to 2^52 apart, and an up that brings
    them back to one size: none is lost.  Multiples of 2^-10 below 2^14, so
    every sum is exact."""
    r = rng(31, M)
    K, n, rank = 64, 3, 8
    a = whole(r, M, K, most=1000 if first == 14 else 2)
    a[:, ::2] = 0
    if first == 14:  # rows without the largest element too
        a[::3, :32] = 0
    b = torch.zeros(K, N, dtype=F16)
    down, up = columns_of_any_size(r, K, n, rank, first, last)
    down[:, 32:, 0] = 0
    up = up.expand(n, rank, N).contiguous() * (1 + torch.from_numpy(r.integers(0, 2, (n, 1, N)))).to(F16)
    pick = torch.from_numpy(r.integers(-1, n, M)).to(torch.int32)
    want, _, _ = lora64(a, b, down, up, pick, None)
    got = lib.gemm_f16f32_lora(a.cuda(), b.cuda(), down.cuda(), up.cuda(), pick.cuda())
    near(got, want, torch.zeros_like(want))


@pytest.mark.parametrize("M,N", LOW_SHAPES)
@pytest.mark.parametrize("rank", [5, 64, 130])
def test_lora_of_any_size_within_its_bound(lib, M, N, rank):
    """The same with no whole numbers, ranks of several blocks and a shared
    product: each element of A . down keeps its 21 bits.  And a row's value
    does not depend on the rows beside it, whichever way they are computed."""
    r = rng(32, M, rank)
    K, n = 100, 3
    a, b = normal(r, M, K), normal(r, K, N, scale=2.0 ** -14)
    a[::3, 0] = 0  # rows without the large elements of column 0
    size = torch.from_numpy(2.0 ** r.integers(-14, 8, rank))
    down = (normal(r, n, K, rank, dtype=torch.float64) * size / size.max()).to(F16)
    up = (normal(r, n, rank, N, dtype=torch.float64) / size[:, None] * 2.0 ** -2).to(F16)
    assert torch.isfinite(up).all()
    down[:, :, 0] = 0
    down[:, 0, 0] = 60000.0
    up[:, 0] = 0
    pick = torch.from_numpy(r.integers(-1, n, M)).to(torch.int32)
    scale = normal(r, n, dtype=F32)
    want, mag, side = lora64(a, b, down, up, pick, scale)
    args = (b.cuda(), down.cuda(), up.cuda())
    got = lib.gemm_f16f32_lora(a.cuda(), *args, pick.cuda(), scale.cuda())
    near(got, want, (K + 2) * U2 * mag + side + want.abs() * 2 * U2)
    other = a.clone()
    other[::2] = normal(r, other[::2].shape[0], K)
    again = lib.gemm_f16f32_lora(other.cuda(), *args, pick.cuda(), scale.cuda())
    assert torch.equal(again[1::2], got[1::2])


@pytest.mark.parametrize("M,N", LOW_SHAPES + [(2200, 3901)])
@pytest.mark.parametrize("rank", [3, 70])
def test_lora_infinities_and_nan(lib, M, N, rank):
    """Infinities and NaN in up and down give the definition's infinities and
    NaN, the same for few rows and many, in their own columns and rows alone."""
    r = rng(33, M, rank)
    K, n = 40, 4
    a, b = whole(r, M, K, most=2), whole(r, K, N)
    down, up = whole(r, n, K, rank, most=1), whole(r, n, rank, N, most=2)
    for e, c, at, x in ((0, 0, 5, float("inf")), (0, rank - 1, 5, float("-inf")), (0, 1, 6, float("-inf")),
                        (1, rank - 1, N - 1, float("inf")), (1, 2, 40, float("nan")), (1, 0, 41, float("inf"))):
        up[e, c, at] = x
    down[2, 7, 1], down[2, 8, 2] = float("inf"), float("-inf")
    pick = torch.from_numpy(r.integers(-1, n, M)).to(torch.int32)
    scale = torch.tensor([1.0, -2.0, 0.5, 0.0])
    want = a.double() @ b.double()
    for t in range(M):
        e = int(pick[t])
        if e >= 0:
            low = (a[t].double()[:, None] * down[e].double()).sum(dim=0)
            want[t] += float(scale[e]) * (low[:, None] * up[e].double()).sum(dim=0)
    got = lib.gemm_f16f32_lora(a.cuda(), b.cuda(), down.cuda(), up.cuda(), pick.cuda(), scale.cuda()).cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    there = ~torch.isnan(want)
    assert torch.isinf(want).any() and torch.equal(got[there], want[there])


# ------------------------------------------------------------------ together

def layer_on(lib, x, ids, w, w1, w2, dy):
    """An expert layer's forward and backward pass through the entry points."""
    E = w1.shape[0]
    offsets, _, slots = lib.tdg_route_plan(ids, E)
    rows = lib.tdg_rows_dispatch(x, slots, torch.zeros(slots.numel(), x.shape[1], dtype=F16, device=x.device))
    h = lib.gemm_f16f32_grouped(rows, w1, offsets, torch.zeros(rows.shape[0], w1.shape[2], device=x.device))
    act = torch.relu(h).to(F16)
    z = lib.gemm_f16f32_grouped(act, w2, offsets, torch.zeros(rows.shape[0], w2.shape[2], device=x.device))
    y = lib.tdg_rows_combine(z, slots, w)
    dz, dw = lib.tdg_rows_combine_grad(dy, z, slots, w, dz=torch.zeros_like(z))
    dz = dz.to(F16)
    dw2 = lib.gemm_f16f32_grouped_tn(act, dz, offsets)
    dact = lib.gemm_f16f32_grouped_nt(dz, w2, offsets, torch.zeros_like(h))
    dh = torch.where(h > 0, dact, torch.zeros_like(dact)).to(F16)
    dw1 = lib.gemm_f16f32_grouped_tn(rows, dh, offsets)
    drows = lib.gemm_f16f32_grouped_nt(dh, w1, offsets, torch.zeros(rows.shape, device=x.device))
    dx = lib.tdg_rows_combine(drows, slots)
    return y, dx, dw, dw1, dw2


def layer_inputs(r, T, k, E, H, F):
    """Whole numbers, so small that every product and sum is exact in FP16
    (rows) and FP32 (sums); some padding tokens without an expert."""
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k]
    ids[-3:] = -1
    sparse = lambda *s: (whole(r, *s, most=1) * torch.from_numpy(r.random(s) < 0.1).to(F16)).cuda()
    return (sparse(T, H), torch.from_numpy(ids).to(torch.int32).cuda(), whole(r, T, k, most=2, dtype=F32).cuda(),
            sparse(E, H, F), sparse(E, F, H), whole(r, T, H, most=1, dtype=F32).cuda())


def test_expert_layer_forward_and_backward(lib):
    r = rng(16)
    T, k, E, H, F = 90, 2, 5, 72, 136
    x, ids, w, w1, w2, dy = layer_inputs(r, T, k, E, H, F)
    got = layer_on(lib, x, ids, w, w1, w2, dy)
    leaf = [t.cpu().double().requires_grad_() for t in (x, w, w1, w2)]
    y = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                y[t] = y[t] + leaf[1][t, j] * (torch.relu(leaf[0][t] @ leaf[2][e]) @ leaf[3][e])
    y.backward(dy.cpu().double())
    for name, g, want in zip(("y", "dx", "dw", "dw1", "dw2"), got, [y.detach()] + [t.grad for t in leaf]):
        assert float(want.abs().max()) < 2048 or name in ("y", "dw", "dx")
        assert torch.equal(g.cpu().double(), want), name


def test_expert_layer_in_a_graph_on_its_own_stream(lib):
    r = rng(17)
    sets = [layer_inputs(r, 80, 2, 6, 64, 96) for _ in range(3)]
    want = [[t.clone() for t in layer_on(lib, *s)] for s in sets]
    held = [t.clone() for t in sets[0]]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer_on(lib, *held)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer_on(lib, *held)
    for s, w in list(zip(sets, want)) * 2:
        for h, t in zip(held, s):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for g, t in zip(got, w):
            assert torch.equal(g, t)
        layer_on(lib, *s)  # eager work between the replays


def test_no_tile_is_read_before_it_lands(lib):
    """With LDS full of NaN at the start (the library's race screen), every
    product is what it is without."""
    r = rng(22)
    off, R = groups_of([300, 40, 0, 513], 0, 0)
    o = off.cuda()
    calls = []
    for K, N in ((256, 264), (200, 65), (40, 40)):
        a, b, dy = normal(r, R, K).cuda(), normal(r, 4, K, N).cuda(), normal(r, R, N).cuda()
        down, up = normal(r, 4, K, 16).cuda(), normal(r, 4, 16, N).cuda()
        pick = torch.from_numpy(r.integers(-1, 4, R)).to(torch.int32).cuda()
        calls += [lambda a=a, b=b: lib.gemm_f16f32_grouped(a, b, o), lambda dy=dy, b=b: lib.gemm_f16f32_grouped_nt(dy, b, o),
                  lambda a=a, dy=dy: lib.gemm_f16f32_grouped_tn(a, dy, o)]
        calls += [lambda m=m, a=a, b=b, d=down, u=up, p=pick: lib.gemm_f16f32_lora(a[:m], b[0], d, u, p[:m])
                  for m in (5, 60, 200, R)]
    plain = [f().clone() for f in calls]
    before = lib.tdg_set_debug_flags(lib.TDG_DEBUG_POISON_LDS)
    try:
        for f, p in zip(calls, plain):
            assert torch.equal(f(), p)
    finally:
        lib.tdg_set_debug_flags(before)


@pytest.mark.parametrize("rows,K,N", GROUPED[16:])
def test_no_large_tile_is_read_before_it_lands(lib, rows, K, N):
    r = rng(28, K, N)
    off, R = groups_of(rows, 0, 0)
    o, G = off.cuda(), len(rows)
    a, b, dy = normal(r, R, K).cuda(), normal(r, G, K, N).cuda(), normal(r, R, N).cuda()
    down, up = normal(r, G, K, 16).cuda(), normal(r, G, 16, N).cuda()
    pick = torch.from_numpy(r.integers(-1, G, R)).to(torch.int32).cuda()
    bt = b.transpose(1, 2).contiguous()
    calls = [lambda: lib.gemm_f16f32_grouped(a, b, o), lambda: lib.gemm_f16f32_grouped_nt(a, bt, o),
             lambda: lib.gemm_f16f32_grouped_tn(a, dy, o), lambda: lib.gemm_f16f32_lora(a, b[0], down, up, pick)]
    plain = [f().clone() for f in calls]
    before = lib.tdg_set_debug_flags(lib.TDG_DEBUG_POISON_LDS)
    try:
        for f, p in zip(calls, plain):
            for _ in range(3):
                assert torch.equal(f(), p)
    finally:
        lib.tdg_set_debug_flags(before)


def test_lora_in_a_graph(lib):
    r = rng(18)
    for M, N in ((4, 96), (300, 96), (500, 4096)):
        a, b = normal(r, M, 128).cuda(), normal(r, 128, N).cuda()
        down, up = normal(r, 3, 128, 8).cuda(), normal(r, 3, 8, N).cuda()
        pick = torch.from_numpy(r.integers(-1, 3, M)).to(torch.int32).cuda()
        ws = torch.empty(lib.tdg_lora_workspace(M, N, 128, 3, 8), dtype=torch.uint8, device="cuda")
        C = torch.empty(M, N, device="cuda")
        lib.gemm_f16f32_lora(a, b, down, up, pick, C=C, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.gemm_f16f32_lora(a, b, down, up, pick, C=C, workspace=ws)
        for i in range(3):
            a.copy_(normal(r, M, 128))
            pick.copy_(torch.from_numpy(r.integers(-1, 3, M)))
            graph.replay()
            torch.cuda.synchronize()
            got = C.clone()
            assert torch.equal(got, lib.gemm_f16f32_lora(a, b, down, up, pick))


def test_two_streams_at_once(lib):
    """Calls with workspaces of their own may overlap."""
    r = rng(19)
    ids = [torch.from_numpy(r.integers(0, 60, (9000, 4))).to(torch.int32).cuda() for _ in range(2)]
    want = [lib.tdg_route_plan(i, 60) for i in ids]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                got[s].append(lib.tdg_route_plan(ids[s], 60))
    torch.cuda.synchronize()
    for s in range(2):
        for g in got[s]:
            assert all(torch.equal(x, y) for x, y in zip(g, want[s]))


def test_wrong_shapes_and_types_are_refused(lib):
    h = torch.zeros(8, 16, dtype=F16, device="cuda")
    w = torch.zeros(2, 16, 4, dtype=F16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    bad = [
        (ValueError, lambda: lib.gemm_f16f32_grouped(h, w, off[:2])),
        (ValueError, lambda: lib.gemm_f16f32_grouped(h[:, :8], w, off)),
        (TypeError, lambda: lib.gemm_f16f32_grouped(h.float(), w, off)),
        (TypeError, lambda: lib.gemm_f16f32_grouped(h, w, off.long())),
        (ValueError, lambda: lib.gemm_f16f32_grouped(h, w, off.cpu())),
        (ValueError, lambda: lib.gemm_f16f32_grouped(h, w.transpose(1, 2), off)),
        (ValueError, lambda: lib.gemm_f16f32_grouped(h, w, off, torch.zeros(8, 5, device="cuda"))),
        (TypeError, lambda: lib.gemm_f16f32_grouped(h, w, off, torch.zeros(8, 4, dtype=F16, device="cuda"))),
        (ValueError, lambda: lib.gemm_f16f32_grouped_tn(h, h[:4], off)),
        (lib.TdgError, lambda: lib.gemm_f16f32_grouped_tn(h, h, off, torch.zeros(1, 16, 16, device="cuda").expand(2, -1, -1))),
        (ValueError, lambda: lib.tdg_rows_dispatch(h, ids[:4])),
        (TypeError, lambda: lib.tdg_rows_dispatch(h.double(), ids)),
        (TypeError, lambda: lib.tdg_rows_dispatch(h, ids, torch.zeros(16, 16, device="cuda"))),
        (ValueError, lambda: lib.tdg_rows_dispatch(h, ids.t().contiguous().t())),
        (ValueError, lambda: lib.tdg_rows_combine(h, ids, torch.ones(8, 3, device="cuda"))),
        (TypeError, lambda: lib.tdg_rows_combine(h, ids, torch.ones(8, 2, dtype=F16, device="cuda"))),
        (ValueError, lambda: lib.tdg_rows_combine_grad(h[:, :8], h, ids)),
        (lib.TdgError, lambda: lib.tdg_rows_combine(h, ids, out=h)),
        (ValueError, lambda: lib.gemm_f16f32_lora(h, w[0], w, w, ids[:, 0].contiguous())),
        (ValueError, lambda: lib.gemm_f16f32_lora(h, w[0], w, torch.zeros(2, 4, 4, dtype=F16, device="cuda"), off)),
        (ValueError, lambda: lib.tdg_route_plan(ids, 4, offsets=off)),
        (lib.TdgError, lambda: lib.tdg_route_plan(ids, 0)),
        (lib.TdgError, lambda: lib.tdg_route_plan(ids, 1025)),
    ]
    for error, fn in bad:
        with pytest.raises(error):
            fn()
