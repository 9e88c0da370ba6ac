"""GPU tests of the layer of experts in every way that its plan cuts the work;
test_layer_cuts_cpu.py asserts that none is left out.  Tolerances as in
test_layer_gpu.py, from the arithmetic alone."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_layer_gpu import F16, F32, F64, U2, lib, near  # noqa: E402,F401

# (tokens, top_k, experts, cols, inner): up thin, with one and with two row tiles, its
# k whole, in two and in four parts, each with every shape of down that goes with it,
# k whole and in two.
CUTS = [(3, 1, 1, 8, 9), (3, 1, 1, 8, 513), (3, 1, 1, 5, 9), (64, 1, 64, 300, 9), (64, 1, 64, 300, 513),
        (4, 2, 8, 4096, 2048), (3, 1, 1, 520, 9), (1, 1, 1, 520, 513), (4, 8, 32, 700, 9), (4, 4, 16, 1500, 513),
        (3, 1, 1, 1025, 9), (1, 1, 1, 1025, 513), (4, 4, 16, 1500, 9), (4, 2, 8, 3001, 513), (3, 1, 1, 8, 1),
        (3, 1, 1, 5, 1), (64, 1, 64, 300, 1), (3, 1, 1, 520, 1), (4, 8, 32, 700, 5), (3, 1, 1, 1025, 7),
        (4, 4, 16, 1500, 3), (12, 1, 1, 8, 9), (12, 1, 1, 8, 513), (12, 1, 1, 5, 70), (64, 4, 24, 3001, 513),
        (64, 4, 24, 1025, 513), (12, 1, 1, 520, 9), (12, 1, 1, 520, 513), (64, 6, 32, 700, 9), (64, 3, 16, 1500, 513),
        (12, 1, 1, 1025, 9), (12, 1, 1, 1025, 513), (64, 1, 6, 4096, 9), (64, 1, 6, 4096, 513), (2, 1, 2, 400, 1100),
        (3, 2, 4, 1100, 5), (3, 2, 4, 5, 70)]

# The same without inner columns: zeros.
EMPTY = [(3, 1, 1, 8), (3, 1, 1, 5), (64, 1, 64, 300), (3, 1, 1, 520), (4, 8, 32, 700), (3, 1, 1, 1025), (4, 4, 16, 1500)]


def problem(T, k, E, cols, inner):
    g = torch.Generator().manual_seed(T + 100 * k + 10000 * E + 1000003 * cols + inner)
    normal = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g) * scale).to(F16)  # noqa: E731
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    return (normal(T, cols), ids, torch.rand(T, k, generator=g), normal(E, cols, 2 * inner, scale=cols ** -0.5),
            normal(E, inner, cols, scale=max(inner, 1) ** -0.5))


def layer64(x, ids, weights, up, down):
    """y in 64 bits, and how far FP32 may be off."""
    T, k = ids.shape
    E, inner, cols = down.shape
    y, tol, size = (torch.zeros(T, cols, dtype=F64) for _ in range(3))
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        a, w, u64, d = x[t].double(), weights[t, j].double()[:, None], up[e].double(), down[e].double()
        b, tb = a @ u64, (cols + 8) * U2 * (a.abs() @ u64.abs())
        g, u, tg, tu = b[:, :inner], b[:, inner:], tb[:, :inner], tb[:, inner:]
        silu = g * torch.sigmoid(g)
        h = silu * u
        th = 1.1 * tg * (u.abs() + tu) + silu.abs() * tu + 8 * U2 * h.abs() + 2.0 ** -120
        z = h @ d
        tz = (inner + 8) * U2 * (h.abs() @ d.abs()) + th @ d.abs() * (1 + inner * U2)
        for of, add in ((y, w * z), (tol, w * tz), (size, w * z.abs())):
            of.index_add_(0, t, add)
    return y, tol + (k + 1) * U2 * size + y.abs() * 2.0 ** -24


@pytest.mark.parametrize("T,k,E,cols,inner", CUTS)
def test_every_plan(lib, T, k, E, cols, inner):  # noqa: F811
    """Workspaces full of NaN, so that what no kernel has written shows."""
    p = problem(T, k, E, cols, inner)
    work = torch.full((lib.tdg_expert_layer_workspace(T, k, E, cols, inner),), 0xFF, dtype=torch.uint8, device="cuda")
    dev = [t.cuda() for t in p]
    got = lib.tdg_expert_layer(*dev, out_dtype=F32, workspace=work)
    near(got, *layer64(*p))
    assert torch.equal(lib.tdg_expert_layer(*dev, out_dtype=F32, workspace=work), got)


@pytest.mark.parametrize("T,k,E,cols", EMPTY)
def test_no_inner_columns_in_every_plan(lib, T, k, E, cols):  # noqa: F811
    x, ids, w, up, down = (t.cuda() for t in problem(T, k, E, cols, 0))
    work = torch.full((lib.tdg_expert_layer_workspace(T, k, E, cols, 0),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full((T, cols), 5.0, device="cuda")
    lib.tdg_expert_layer(x, ids, w, up, down, out=y, workspace=work)
    assert (y == 0).all()
