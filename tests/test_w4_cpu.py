"""CPU tests of the 4-bit weights and of the layer of experts for a few tokens:
every refusal comes before any HIP call, empty calls need no device, and the
workspace sizes are what the header says.  Addresses here are made up; nothing
is launched."""
import ctypes

import pytest

import tiled_dense_gemm_loop_amd as tdg
from conftest import no_device_only

BAD, OK, NODEV = tdg.TDG_ERR_INVALID_ARG, tdg.TDG_OK, tdg.TDG_ERR_NO_DEVICE
TOO_BIG = tdg.TDG_ERR_UNSUPPORTED
G = 1 << 30  # addresses a gibibyte apart never overlap here
A, B, C, D, E, F, H, I = (G * i for i in range(1, 9))


def call(name, args, **change):
    """Calls `name` with a dict of arguments, some of them changed."""
    assert not set(change) - set(args), set(change) - set(args)
    return getattr(tdg.load_library(), name)(*{**args, **change}.values(), None)


# 3 matrices of 200 x 96: 2 blocks of 96 pieces, groups of 64: 4 of them
QUANT = dict(count=3, K=200, N=96, group=64, w=A, ldw=96, stride_w=200 * 96, codes=B, ld_codes=96, stride_codes=192,
             scales=C, ld_scales=96, stride_scales=384, zeros=D, ld_zeros=96, stride_zeros=384)
DEQUANT = dict(elem=0, count=3, K=200, N=96, group=64, codes=B, ld_codes=96, stride_codes=192, scales=C, ld_scales=96,
               stride_scales=384, zeros=D, ld_zeros=96, stride_zeros=384, w=A, ldw=96, stride_w=200 * 96)
W4 = dict(M=5, N=96, K=200, group=64, a=A, lda=200, codes=B, ld_codes=96, scales=C, ld_scales=96, zeros=D,
          ld_zeros=96, c=E, ldc=96)
W4G = dict(groups=3, offsets=F, M=5, N=96, K=200, group=64, a=A, lda=200, codes=B, ld_codes=96, stride_codes=192,
           scales=C, ld_scales=96, stride_scales=384, zeros=D, ld_zeros=96, stride_zeros=384, c=E, ldc=96)
LAYER = dict(elem=0, tokens=5, top_k=2, experts=4, cols=64, inner=32, x=A, ldx=64, ids=B, ld_ids=2, weights=C,
             ld_weights=2, up=D, ld_up=64, stride_up=4096, down=E, ld_down=64, stride_down=2048, y=F, ldy=64, ws=H,
             ws_bytes=1 << 20)

FAR = 1 << 62
SHARED = [dict(K=-1), dict(N=-1), dict(group=0), dict(group=16), dict(group=48), dict(group=-32), dict(ld_codes=95),
          dict(ld_scales=95), dict(ld_zeros=95), dict(codes=None), dict(scales=None), dict(codes=B + 8),
          dict(scales=C + 1), dict(ld_codes=FAR), dict(ld_scales=FAR), dict(ld_zeros=FAR), dict(K=1 << 31),
          dict(N=1 << 31)]
STACKED = [dict(stride_codes=-1), dict(stride_scales=-1), dict(stride_zeros=-1), dict(stride_codes=FAR)]
REFUSED = [
    ("tdg_w4_quantize", QUANT, SHARED + STACKED + [
        dict(count=-1), dict(w=None), dict(w=A + 1), dict(ldw=95), dict(ldw=FAR), dict(stride_w=-1),
        dict(codes=A), dict(scales=A), dict(zeros=A), dict(scales=B), dict(zeros=B), dict(zeros=C),
        dict(codes=A + 2 * 3 * 200 * 96 - 16), dict(stride_codes=191), dict(stride_scales=383),
        dict(stride_zeros=383)]),
    ("tdg_w4_dequantize", DEQUANT, SHARED + STACKED + [
        dict(elem=2), dict(elem=-1), dict(count=-1), dict(w=None), dict(w=A + 1), dict(elem=1, w=A + 2), dict(ldw=95),
        dict(ldw=FAR), dict(stride_w=200 * 96 - 1), dict(w=B), dict(w=C), dict(w=D)]),
    ("gemm_f16w4f32", W4, SHARED + [
        dict(M=-1), dict(M=1 << 31), dict(a=None), dict(a=A + 1), dict(lda=199), dict(lda=FAR), dict(c=None),
        dict(c=E + 2), dict(ldc=95), dict(ldc=FAR), dict(c=A), dict(c=B), dict(c=C), dict(c=D)]),
    ("gemm_f16w4f32_grouped", W4G, SHARED + STACKED + [
        dict(groups=-1), dict(groups=1025), dict(offsets=None), dict(offsets=F + 2), dict(M=-1), dict(M=1 << 31),
        dict(a=None), dict(a=A + 1), dict(lda=199), dict(lda=FAR), dict(c=None), dict(c=E + 2), dict(ldc=95),
        dict(ldc=FAR), dict(c=A), dict(c=B), dict(c=C), dict(c=D), dict(c=F), dict(c=B + 64 * 2 * 192)]),
    ("tdg_expert_layer", LAYER, [
        dict(elem=2), dict(elem=-1), dict(tokens=-1), dict(top_k=0), dict(top_k=-1), dict(experts=0),
        dict(experts=1025), dict(cols=-1), dict(inner=-1), dict(cols=1 << 30), dict(inner=1 << 30), dict(ldx=63),
        dict(ld_ids=1), dict(ld_weights=1), dict(ld_up=63), dict(ld_down=63), dict(ldy=63), dict(x=None),
        dict(ids=None), dict(up=None), dict(down=None), dict(y=None), dict(x=A + 1), dict(ids=B + 2),
        dict(weights=C + 2), dict(up=D + 1), dict(down=E + 1), dict(y=F + 1), dict(elem=1, y=F + 2), dict(y=A),
        dict(y=B), dict(y=C), dict(y=D), dict(y=E), dict(stride_up=-1), dict(stride_down=-1), dict(stride_up=FAR),
        dict(ldx=FAR), dict(ldy=FAR), dict(ws=None), dict(ws=H + 8), dict(ws_bytes=100), dict(ws=A), dict(ws=B),
        dict(ws=C), dict(ws=D), dict(ws=E), dict(ws=F)]),
]
CASES = [(n, args, ch) for n, args, changes in REFUSED for ch in changes]


@pytest.mark.parametrize("name,args,change", CASES, ids=["%s %s" % (n, c) for n, _, c in CASES])
def test_refused_before_the_device(name, args, change):
    assert call(name, args, **change) == BAD


@no_device_only
@pytest.mark.parametrize("name,args", [(n, a) for n, a, _ in REFUSED], ids=[n for n, _, _ in REFUSED])
def test_sound_arguments_reach_the_device_check(name, args):
    assert call(name, args) == NODEV


@no_device_only
def test_what_may_be_left_out():
    for name, args in (("tdg_w4_quantize", QUANT), ("tdg_w4_dequantize", DEQUANT), ("gemm_f16w4f32_grouped", W4G)):
        assert call(name, args, zeros=None, ld_zeros=0, stride_zeros=0) == NODEV
    assert call("gemm_f16w4f32", W4, zeros=None, ld_zeros=0) == NODEV
    assert call("gemm_f16w4f32", W4, group=1 << 20, ld_scales=96) == NODEV  # one group for all of k
    assert call("gemm_f16w4f32", W4, K=0, a=None, codes=None, scales=None) == NODEV  # zeros in C
    assert call("gemm_f16w4f32_grouped", W4G, stride_codes=0, stride_scales=0, stride_zeros=0) == NODEV
    assert call("tdg_expert_layer", LAYER, weights=None, ld_weights=0) == NODEV
    assert call("tdg_expert_layer", LAYER, inner=0, up=None, down=None) == NODEV  # zeros in y


def test_empty_calls_need_no_device():
    assert call("tdg_w4_quantize", QUANT, count=0, w=None, codes=None, scales=None, zeros=None) == OK
    assert call("tdg_w4_quantize", QUANT, K=0, codes=None) == OK
    assert call("tdg_w4_dequantize", DEQUANT, N=0, w=None) == OK
    assert call("gemm_f16w4f32", W4, M=0, a=None, c=None) == OK
    assert call("gemm_f16w4f32", W4, N=0, c=None, codes=None) == OK
    assert call("gemm_f16w4f32_grouped", W4G, groups=0, offsets=None, codes=None, scales=None) == OK
    assert call("gemm_f16w4f32_grouped", W4G, M=0, a=None, c=None) == OK
    assert call("tdg_expert_layer", LAYER, tokens=0, x=None, ids=None, y=None, ws=None) == OK
    assert call("tdg_expert_layer", LAYER, cols=0, x=None, y=None, ws=None) == OK


def test_more_than_a_few_tokens_are_refused():
    most, k = tdg.TDG_LAYER_MAX_TOKENS, tdg.TDG_LAYER_MAX_TOP_K
    assert (most, k) == (64, 32)
    assert call("tdg_expert_layer", LAYER, tokens=most + 1) == TOO_BIG
    assert call("tdg_expert_layer", LAYER, top_k=k + 1, ld_ids=k + 1, ld_weights=k + 1) == TOO_BIG
    with pytest.raises(tdg.TdgError):
        tdg.tdg_expert_layer_workspace(most + 1, 1, 8, 64, 64)


def test_grids_past_one_launch_are_refused():
    far = [i << 55 for i in range(1, 8)]
    n = 1 << 30
    assert call("gemm_f16w4f32", W4, M=1 << 30, N=n, K=32, a=far[0], lda=32, codes=far[1], ld_codes=n, scales=far[2],
                ld_scales=n, zeros=None, c=1 << 62, ldc=n) == TOO_BIG
    places = dict(w=far[0], codes=far[1], scales=far[2], zeros=far[3])
    one = dict(count=1, N=1, ldw=1, ld_codes=1, ld_scales=1, ld_zeros=1)
    for name, args in (("tdg_w4_quantize", QUANT), ("tdg_w4_dequantize", DEQUANT)):
        assert call(name, args, count=65536, **places) == TOO_BIG
        assert call(name, args, **{**one, **places}, K=65535 * 128 + 1) == TOO_BIG
    assert call("tdg_w4_quantize", QUANT, **{**one, **places}, K=65535 * 96 + 1, group=96) == TOO_BIG


@no_device_only
def test_the_limits_that_the_header_states():
    """The largest counts that quantize and dequantize take."""
    far = [i << 55 for i in range(1, 8)]
    places = dict(w=far[0], codes=far[1], scales=far[2], zeros=far[3])
    one = dict(count=1, N=1, ldw=1, ld_codes=1, ld_scales=1, ld_zeros=1)
    for name, args in (("tdg_w4_quantize", QUANT), ("tdg_w4_dequantize", DEQUANT)):
        assert call(name, args, count=65535, **places) == NODEV
        assert call(name, args, **{**one, **places}, K=65535 * 128) == NODEV
    assert call("tdg_w4_quantize", QUANT, **{**one, **places}, K=65535 * 96, group=96) == NODEV


def test_workspace_sizes():
    assert tdg.tdg_expert_layer_workspace(0, 1, 8, 64, 64) == 0
    small, large = (tdg.tdg_expert_layer_workspace(t, 8, 128, 2048, 768) for t in (1, 64))
    assert 8 * (768 + 2048) * 4 <= small <= large <= 64 << 20
    for bad in ((-1, 1, 8, 8, 8), (1, 0, 8, 8, 8), (1, 1, 0, 8, 8), (1, 1, 8, -1, 8), (1, 1, 8, 8, 1 << 30)):
        with pytest.raises(tdg.TdgError):
            tdg.tdg_expert_layer_workspace(*bad)
    null = ctypes.POINTER(ctypes.c_size_t)()
    assert tdg.load_library().tdg_expert_layer_workspace(1, 1, 1, 1, 1, null) == BAD


def test_host_tensors_and_wrong_types_are_refused():
    import torch
    h = torch.zeros(4, 256, dtype=torch.float16)
    codes, scales = torch.zeros(2, 8, 64, dtype=torch.uint8), torch.zeros(2, 8, dtype=torch.float16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for fn in (lambda: tdg.tdg_w4_quantize(h), lambda: tdg.tdg_w4_quantize(h[None]),
               lambda: tdg.tdg_w4_dequantize(codes, scales), lambda: tdg.gemm_f16w4f32(h, codes, scales),
               lambda: tdg.gemm_f16w4f32_grouped(h, codes[None], scales[None], ids[0]),
               lambda: tdg.tdg_expert_layer(h, ids, None, h[None], h[None])):
        with pytest.raises(ValueError, match="device tensor"):
            fn()
    for fn in (lambda: tdg.tdg_w4_quantize(h.float()), lambda: tdg.gemm_f16w4f32(h.float(), codes, scales),
               lambda: tdg.tdg_expert_layer(h.float(), ids, None, h[None], h[None])):
        with pytest.raises(TypeError):
            fn()


# (what, group, the most columns of 65535 matrices of one block, and of 16 of 4095)
MOST_COLUMNS = [("tdg_w4_quantize", QUANT, 64, 64 * 256, 64 * 256), ("tdg_w4_quantize", QUANT, 96, 64 * 256, 64 * 192),
                ("tdg_w4_dequantize", DEQUANT, 64, 128 * 256, 128 * 256)]


def _columns(args, count, K, N, group):
    """The arguments for `count` dense matrices of K x N, each array far from the others."""
    blocks, groups = -(-K // 128), -(-K // group)
    return dict(args, count=count, K=K, N=N, group=group, w=1 << 55, ldw=N, stride_w=K * N, codes=2 << 55, ld_codes=N,
                stride_codes=blocks * N, scales=3 << 55, ld_scales=N, stride_scales=groups * N, zeros=4 << 55,
                ld_zeros=N, stride_zeros=groups * N)


@pytest.mark.parametrize("name,args,group,one,many", MOST_COLUMNS)
def test_more_columns_than_a_launch_holds_are_refused(name, args, group, one, many):
    K = 128 if group == 64 else 96
    assert call(name, _columns(args, 65535, K, one + 1, group)) == TOO_BIG
    assert call(name, _columns(args, 16, 4095 * 128, many + 1, group)) == TOO_BIG


@no_device_only
@pytest.mark.parametrize("name,args,group,one,many", MOST_COLUMNS)
def test_as_many_columns_as_a_launch_holds_are_taken(name, args, group, one, many):
    K = 128 if group == 64 else 96
    assert call(name, _columns(args, 65535, K, one, group)) == NODEV
    assert call(name, _columns(args, 16, 4095 * 128, many, group)) == NODEV
