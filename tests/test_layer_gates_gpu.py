"""GPU tests of the layer of experts where the gate is so far below zero that
exp(-gate) passes FP32's largest value, and silu(gate) times the other half
does not vanish.

Each sum here has one term that is not zero, so h is the only inexact step
before y: two exponentials within 2 ulp (2^-22 relative each, as a quotient of
them would be) and three products, below 2^-20 together; the down product and
the weight of 1 add a rounding each, y's sum none."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

F16, F32 = torch.float16, torch.float32
BIG = 60000.0


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import tiled_dense_gemm_loop_amd as t
    t.load_library()
    return t


def problem(gates, cols, experts=1):
    """One token with x = (1, BIG, 0 ...): column i of up gives the gate
    gates[i] and BIG * BIG beside it, row i of down BIG in column i."""
    inner = len(gates)
    x = torch.zeros(1, cols, dtype=F16)
    x[0, 0], x[0, 1] = 1, BIG
    up, down = torch.zeros(experts, cols, 2 * inner, dtype=F16), torch.zeros(experts, inner, cols, dtype=F16)
    up[:, 0, :inner] = torch.tensor(gates, dtype=F16)
    up[:, 1, inner:] = BIG
    for i in range(inner):
        down[:, i, i] = BIG
    return x, torch.zeros(1, 1, dtype=torch.int32), up, down


GATES = [-60.0, -80.0, -86.9375, -87.0, -87.0625, -88.0, -88.6875, -88.75, -89.0, -90.0, -95.0, -100.0, -103.0, -104.0,
         -108.0, -112.0, 0.0, 5.0, 90.0, 300.0]


# whole k of the up product, in two and in four parts (which down joins)
@pytest.mark.parametrize("cols", [64, 600, 1100])
def test_gates_far_below_zero(lib, cols):
    x, ids, up, down = problem(GATES, cols)
    y = lib.tdg_expert_layer(x.cuda(), ids.cuda(), None, up.cuda(), down.cuda(), out_dtype=F32).cpu().double()
    big = float(torch.tensor(BIG, dtype=F16))
    for i, g in enumerate(GATES):
        want = g / (1 + math.exp(-g)) * big * big * big  # (in 64 bits; big is exact)
        got = float(y[0, i])
        # h itself may be a subnormal of FP32: half a step of it, times down
        assert abs(got - want) <= 2.0 ** -19 * abs(want) + 2.0 ** -150 * big, (g, got, want)


@pytest.mark.parametrize("cols", [64, 600])
def test_an_infinity_beside_a_gate_far_below_zero(lib, cols):
    """-100 / (1 + exp(100)) is a number below zero, and times infinity it is
    -infinity; where the gate is -infinity there is no value."""
    gates = [-100.0, -88.75, -50.0, 50.0, float("-inf"), float("inf")]
    x, ids, up, down = problem(gates, cols)
    inner = len(gates)
    out = []
    for i in range(inner):
        down.zero_()
        down[:, i, 0] = 1
        for j in range(inner):  # one element of h at a time: the others' columns are made zeros
            if j != i:
                up[:, 0, j], up[:, 0, inner + j], up[:, 1, inner + j] = 0, 0, 0
            else:
                up[:, 0, j], up[:, 0, inner + j], up[:, 1, inner + j] = gates[j], float("inf"), BIG
        y = lib.tdg_expert_layer(x.cuda(), ids.cuda(), None, up.cuda(), down.cuda(), out_dtype=F32)
        out.append(float(y[0, 0]))
    inf = float("inf")
    assert out[:4] == [-inf, -inf, -inf, inf] and math.isnan(out[4]) and out[5] == inf, out
