"""CPU tests of the operators whose rows pick their weights: every refusal
comes before any HIP call, empty calls need no device, and the workspace
sizes are what the header says.  Addresses here are made up; nothing is
launched."""
import ctypes

import pytest

import tiled_dense_gemm_loop_amd as tdg
from conftest import no_device_only

BAD, OK, NODEV = tdg.TDG_ERR_INVALID_ARG, tdg.TDG_OK, tdg.TDG_ERR_NO_DEVICE
TOO_BIG = tdg.TDG_ERR_UNSUPPORTED
G = 1 << 30  # addresses a gibibyte apart never overlap here
A, B, C, D, E, F = (G * i for i in range(1, 7))


def call(name, args, **change):
    """Calls `name` with a dict of arguments, some of them changed."""
    assert not set(change) - set(args), set(change) - set(args)
    return getattr(tdg.load_library(), name)(*{**args, **change}.values(), None)


PLAN = dict(tokens=100, top_k=2, experts=8, ids=A, ld_ids=2, offsets=B, order=C, slots=D, ws=None, ws_bytes=0)
DISPATCH = dict(elem=0, tokens=10, top_k=2, cols=64, x=A, ldx=64, slots=B, rows=20, out=C, ldo=64)
COMBINE = dict(row_elem=1, token_elem=0, tokens=10, top_k=2, cols=64, z=A, ldz=64, rows=20, slots=B, weights=C,
               ld_weights=2, y=D, ldy=64)
GRAD = dict(row_elem=1, token_elem=1, tokens=10, top_k=2, cols=64, dy=A, ldy=64, z=B, ldz=64, rows=20, slots=C,
            weights=D, ld_weights=2, dz=E, lddz=64, dweights=F, ld_dweights=2)
NN = dict(groups=4, offsets=A, M=64, N=32, K=16, a=B, lda=16, b=C, ldb=32, stride_b=512, c=D, ldc=32)
NT = dict(groups=4, offsets=A, M=64, N=32, K=16, a=B, lda=16, b=C, ldb=16, stride_b=512, c=D, ldc=32)
TN = dict(groups=4, offsets=A, rows=64, M=16, N=32, a=B, lda=16, b=C, ldb=32, c=D, ldc=32, stride_c=512)
LORA = dict(M=8, N=64, K=32, a=A, lda=32, b=B, ldb=64, adapters=3, rank=4, down=C, ld_down=4, stride_down=128,
            up=D, ld_up=64, stride_up=256, adapter=E, scale=E + 4096, c=F, ldc=64, ws=F + (1 << 20),
            ws_bytes=1 << 24)

FAR = 1 << 62
REFUSED = [
    ("tdg_route_plan", PLAN, [
        dict(tokens=-1), dict(top_k=0), dict(experts=0), dict(experts=1025), dict(tokens=1 << 30, top_k=2),
        dict(ld_ids=1), dict(ids=None), dict(offsets=None), dict(order=None), dict(slots=None), dict(ids=A + 2),
        dict(offsets=B + 1), dict(slots=C + 4), dict(order=A), dict(offsets=D), dict(ld_ids=FAR),
        dict(tokens=4097, top_k=1), dict(tokens=4097, top_k=1, ws=E, ws_bytes=63),
        dict(tokens=4097, top_k=1, ws=C, ws_bytes=4096), dict(tokens=4097, top_k=1, ws=E + 2, ws_bytes=4096)]),
    ("tdg_rows_dispatch", DISPATCH, [
        dict(elem=2), dict(elem=-1), dict(tokens=-1), dict(top_k=0), dict(cols=-1), dict(rows=-1), dict(ldx=63),
        dict(ldo=63), dict(x=None), dict(out=None), dict(slots=None), dict(out=A), dict(out=B), dict(x=A + 1),
        dict(out=C + 1), dict(slots=B + 2), dict(elem=1, x=A + 2), dict(ldx=FAR), dict(ldo=FAR),
        dict(tokens=1 << 30, top_k=2), dict(rows=1 << 31)]),
    ("tdg_rows_combine", COMBINE, [
        dict(row_elem=2), dict(token_elem=7), dict(tokens=-1), dict(top_k=0), dict(ldz=63), dict(ldy=63),
        dict(ld_weights=1), dict(z=None), dict(y=None), dict(slots=None), dict(y=A), dict(y=B), dict(y=C),
        dict(z=A + 2), dict(y=D + 1), dict(weights=C + 2), dict(ldz=FAR)]),
    ("tdg_rows_combine_grad", GRAD, [
        dict(row_elem=2), dict(token_elem=-1), dict(tokens=-1), dict(top_k=0), dict(ldy=63), dict(ldz=63),
        dict(lddz=63), dict(ld_weights=1), dict(ld_dweights=1), dict(dy=None), dict(z=None), dict(dz=None),
        dict(dweights=None), dict(slots=None), dict(dz=A), dict(dz=B), dict(dz=C), dict(dz=D), dict(dz=F),
        dict(dweights=A), dict(dweights=B), dict(dweights=D), dict(dz=E + 2), dict(dweights=F + 2)]),
    ("gemm_f16f32_grouped", NN, [
        dict(groups=-1), dict(groups=1025), dict(offsets=None), dict(offsets=A + 2), dict(M=-1), dict(N=-1),
        dict(K=-1), dict(lda=15), dict(ldb=31), dict(ldc=31), dict(a=None), dict(b=None), dict(c=None),
        dict(c=B), dict(c=C), dict(c=A), dict(c=C + 2 * 1024), dict(a=B + 1), dict(b=C + 1), dict(c=D + 2),
        dict(stride_b=-1), dict(stride_b=FAR), dict(lda=FAR), dict(M=1 << 31)]),
    ("gemm_f16f32_grouped_nt", NT, [
        dict(groups=-1), dict(offsets=None), dict(lda=15), dict(ldb=15), dict(ldc=31), dict(a=None), dict(b=None),
        dict(c=None), dict(c=B), dict(c=C), dict(stride_b=-1), dict(N=1 << 31)]),
    ("gemm_f16f32_grouped_tn", TN, [
        dict(groups=-1), dict(offsets=None), dict(lda=15), dict(ldb=31), dict(ldc=31), dict(a=None), dict(b=None),
        dict(c=None), dict(c=B), dict(c=C), dict(stride_c=511), dict(stride_c=-1), dict(rows=-1)]),
    ("gemm_f16f32_lora", LORA, [
        dict(M=-1), dict(lda=31), dict(ldb=63), dict(ldc=63), dict(adapters=-1), dict(rank=-1), dict(rank=257),
        dict(ld_down=3), dict(ld_up=63), dict(stride_down=-1), dict(stride_up=-1), dict(down=None), dict(up=None),
        dict(adapter=None), dict(adapter=E + 2), dict(scale=E + 4097), dict(a=A + 1), dict(up=D + 1), dict(c=C),
        dict(c=D), dict(c=E), dict(ws=None), dict(ws_bytes=3), dict(ws=F + (1 << 20) + 8), dict(ws=F), dict(ws=A),
        dict(ws=C), dict(ws=E)]),
]
CASES = [(n, args, ch) for n, args, changes in REFUSED for ch in changes]


@pytest.mark.parametrize("name,args,change", CASES, ids=["%s %s" % (n, c) for n, _, c in CASES])
def test_refused_before_the_device(name, args, change):
    assert call(name, args, **change) == BAD


@no_device_only
@pytest.mark.parametrize("name,args", [(n, a) for n, a, _ in REFUSED], ids=[n for n, _, _ in REFUSED])
def test_sound_arguments_reach_the_device_check(name, args):
    assert call(name, args) == NODEV


def test_empty_calls_need_no_device():
    assert call("tdg_rows_dispatch", DISPATCH, tokens=0) == OK
    assert call("tdg_rows_dispatch", DISPATCH, cols=0) == OK
    assert call("tdg_rows_dispatch", DISPATCH, rows=0, out=None) == OK
    assert call("tdg_rows_combine", COMBINE, tokens=0) == OK
    assert call("tdg_rows_combine", COMBINE, cols=0) == OK
    assert call("tdg_rows_combine_grad", GRAD, tokens=0) == OK
    assert call("gemm_f16f32_grouped", NN, groups=0, offsets=None, b=None) == OK
    assert call("gemm_f16f32_grouped", NN, M=0, a=None, c=None) == OK
    assert call("gemm_f16f32_grouped_nt", NT, N=0, b=None, c=None) == OK
    assert call("gemm_f16f32_grouped_tn", TN, M=0, a=None, c=None) == OK
    assert call("gemm_f16f32_grouped_tn", TN, groups=0, offsets=None, c=None) == OK
    assert call("gemm_f16f32_lora", LORA, M=0, a=None, c=None, adapter=None) == OK
    assert call("gemm_f16f32_lora", LORA, N=0, ws=None) == OK


@no_device_only
def test_adapter_arguments_are_not_needed_without_adapters():
    none = dict(down=None, up=None, adapter=None, scale=None, ws=None, ws_bytes=0)
    assert call("gemm_f16f32_lora", LORA, adapters=0, **none) == NODEV
    assert call("gemm_f16f32_lora", LORA, rank=0, **none) == NODEV
    assert call("tdg_rows_combine", COMBINE, weights=None, ld_weights=0) == NODEV
    assert call("gemm_f16f32_grouped", NN, stride_b=0) == NODEV  # one B for all groups


def test_grids_past_one_launch_are_refused():
    """Sizes that pass every check but would need more workgroups than one
    launch counts, in any of a call's launches."""
    far = [1 << 50, 2 << 50, 3 << 50, 4 << 50, 5 << 50, 6 << 50, 7 << 50]
    M = (1 << 26) + 4  # the launch that cuts low's rows has a workgroup for four
    big = dict(K=1, rank=1, a=far[0], lda=1, b=far[1], down=far[2], ld_down=1, stride_down=1, up=far[3],
               adapter=far[4], c=far[5], ws=far[6], ws_bytes=1 << 45)
    for size in (dict(M=M, N=1), dict(M=1 << 20, N=1 << 20)):
        n = size["N"]
        assert call("gemm_f16f32_lora", LORA, **{**big, **size}, ldb=n, ld_up=n, stride_up=n, ldc=n) == TOO_BIG
    n = 1 << 25  # few rows: 65536 workgroups across at the join
    assert call("gemm_f16f32_lora", LORA, **big, M=4, N=n + 1, ldb=n + 1, ld_up=n + 1, stride_up=n + 1,
                ldc=n + 1) == TOO_BIG
    assert call("tdg_rows_dispatch", DISPATCH, tokens=1 << 24, top_k=1, cols=8192, ldx=8192, ldo=8192, rows=1,
                x=far[0], out=far[1], slots=far[2]) == TOO_BIG
    m = 1 << 30
    for name, args, more in (("gemm_f16f32_grouped", NN, dict(lda=1, ldb=m, stride_b=m)),
                             ("gemm_f16f32_grouped_nt", NT, dict(lda=1, ldb=1, stride_b=m))):
        assert call(name, args, M=m, N=m, K=1, ldc=m, offsets=far[3], a=far[0], b=far[1], c=1 << 62, groups=1,
                    **more) == TOO_BIG


@no_device_only
def test_the_limits_that_the_header_states():
    """The largest top_k and N are taken, the next ones refused."""
    far = [i << 50 for i in range(1, 8)]
    grad = dict(tokens=1, cols=1, ldy=1, ldz=1, lddz=1, rows=1, dy=far[0], z=far[1], slots=far[2], weights=far[3],
                dz=far[4], dweights=far[5])
    for top_k, rc in ((524280, NODEV), (524281, TOO_BIG)):
        assert call("tdg_rows_combine_grad", GRAD, **grad, top_k=top_k, ld_weights=top_k, ld_dweights=top_k) == rc
    for n, rc in ((33553920, NODEV), (33553921, TOO_BIG)):
        assert call("gemm_f16f32_lora", LORA, M=1, N=n, K=1, rank=1, a=far[0], lda=1, b=far[1], ldb=n, down=far[2],
                    ld_down=1, stride_down=1, up=far[3], ld_up=n, stride_up=n, adapter=far[4], c=far[5], ldc=n,
                    ws=far[6], ws_bytes=1 << 45) == rc


def test_workspace_sizes():
    assert tdg.tdg_route_workspace(0, 1, 8) == 0
    assert tdg.tdg_route_workspace(512, 8, 1024) == 0
    assert 2 * 8 * 4 <= tdg.tdg_route_workspace(4097, 1, 8) <= 1 << 20
    assert tdg.tdg_route_workspace(1 << 27, 8, 1024) <= 1 << 20
    for bad in ((-1, 1, 8), (1, 0, 8), (1, 1, 0), (1, 1, 1025), (1 << 30, 2, 8)):
        with pytest.raises(tdg.TdgError):
            tdg.tdg_route_workspace(*bad)
    assert tdg.tdg_lora_workspace(0, 64, 64, 4, 16) == 0
    assert tdg.tdg_lora_workspace(4, 64, 64, 4, 16) >= 4 * 16 * 4
    for bad in ((-1, 1, 1, 1, 1), (1, 1, 1, 1, 257), (1, 1, 1, -1, 1)):
        with pytest.raises(tdg.TdgError):
            tdg.tdg_lora_workspace(*bad)
    assert tdg.load_library().tdg_lora_workspace(1, 1, 1, 1, 1, ctypes.POINTER(ctypes.c_size_t)()) == BAD


def test_host_tensors_are_refused():
    import torch
    x = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    h = torch.zeros(4, 8, dtype=torch.float16)
    for fn in (lambda: tdg.tdg_route_plan(i, 4), lambda: tdg.tdg_rows_dispatch(x, i),
               lambda: tdg.tdg_rows_combine(x, i), lambda: tdg.tdg_rows_combine_grad(x, x, i),
               lambda: tdg.gemm_f16f32_grouped(h, h[None], i[0]),
               lambda: tdg.gemm_f16f32_grouped_nt(h, h[None], i[0]),
               lambda: tdg.gemm_f16f32_grouped_tn(h, h, i[0]),
               lambda: tdg.gemm_f16f32_lora(h, h, h[None], h[None], i[0])):
        with pytest.raises(ValueError, match="device tensor"):
            fn()
    with pytest.raises(TypeError):
        tdg.tdg_route_plan(i.long(), 4)
