"""The experts' bf16 products and gradients and the 4-bit products without a GPU:
every bad argument of the C ABI and of the binding is refused before anything is
launched."""
import ctypes
import os

import pytest
import torch

from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH),
                                reason="libqmoe.so not built (run __graft_entry__.build())")
OK, INV, UNS = ops.QMOE_OK, ops.QMOE_ERR_INVALID_ARG, ops.QMOE_ERR_UNSUPPORTED
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def _caller(name, **base):
    """A call of `name` with the arguments `base` (in order), some replaced."""
    fn = getattr(ops.lib(), name)

    def call(**kw):
        assert set(kw) <= set(base)
        return fn(*{**base, **kw}.values())
    return call


def test_grouped_matmul_refusals():
    c = _caller("qmoe_grouped_matmul", a=P, pair_rows=0, b=P, trans=0, srt=P, te=P, off=P, npad=P,
                T=4, k=2, E=8, block_m=16, N=64, K=256, act=0, gu=None, out=P, out_dtype=0,
                stream=None)
    for bad in (dict(pair_rows=2), dict(trans=-1), dict(T=-1), dict(k=0), dict(k=9), dict(E=0),
                dict(block_m=48), dict(T=1 << 30), dict(N=0), dict(K=0), dict(act=3), dict(act=-1),
                dict(act=1, trans=1), dict(act=2), dict(act=2, trans=1), dict(gu=P),
                dict(out_dtype=2), dict(a=None), dict(b=None), dict(srt=None), dict(te=None),
                dict(off=None), dict(npad=None), dict(out=None), dict(a=ODD), dict(b=ODD),
                dict(out=ODD), dict(act=1, gu=ODD)):
        assert c(**bad) == INV, bad
    for big in (dict(E=1025, k=2), dict(N=60), dict(K=260), dict(act=1, N=72),
                dict(N=(1 << 22) + 8), dict(K=(1 << 22) + 8), dict(N=1 << 20, K=2048),
                dict(T=1 << 20, K=2048), dict(T=1 << 19, K=2048, pair_rows=1),
                dict(trans=1, N=1 << 20, K=2048)):
        assert c(**big) == UNS, big
    assert c(T=0, a=None) == OK


def test_grouped_wgrad_refusals():
    c = _caller("qmoe_grouped_wgrad", dy=P, x=P, pair_rows=0, srt=P, off=P, T=4, k=2, E=8,
                block_m=16, N=64, K=256, dw=P, out_dtype=1, accumulate=0, stream=None)
    for bad in (dict(pair_rows=2), dict(T=-1), dict(k=0), dict(k=9), dict(E=0), dict(block_m=8),
                dict(T=1 << 30), dict(N=0), dict(K=0), dict(out_dtype=2), dict(accumulate=2),
                dict(accumulate=1, out_dtype=0), dict(dy=None), dict(x=None), dict(srt=None),
                dict(off=None), dict(dw=None), dict(dy=ODD), dict(x=ODD), dict(dw=ODD)):
        assert c(**bad) == INV, bad
    for big in (dict(E=1025), dict(N=60), dict(K=260), dict(N=(1 << 22) + 8), dict(K=(1 << 22) + 8),
                dict(T=1 << 20, K=2048), dict(T=1 << 19, N=2048)):
        assert c(**big) == UNS, big


def test_combine_backward_refusals():
    c = _caller("qmoe_combine_backward", dout=P, y=P, dtype=0, ids=P, w=P, T=4, k=2, H=64, E=8,
                add=None, dy=P, dw=P, dz=P, stream=None)
    for bad in (dict(dtype=2), dict(T=-1), dict(k=0), dict(k=9), dict(k=17, E=64), dict(E=0),
                dict(H=0), dict(H=60), dict(T=1 << 30), dict(add=P, dz=None), dict(dout=None),
                dict(y=None), dict(ids=None), dict(w=None), dict(dy=None), dict(dout=ODD),
                dict(y=ODD), dict(dy=ODD)):
        assert c(**bad) == INV, bad
    assert c(E=1025) == UNS
    assert c(T=0, dout=None) == OK


def test_w4_matmul_refusals():
    c = _caller("qmoe_w4_matmul", x=P, codes=P, scale=P, fmt=0, group=32, M=4, N=64, K=256, act=0,
                add=None, out=P, out_dtype=0, ws=P, ws_bytes=1 << 40, stream=None)
    for bad in (dict(fmt=2), dict(fmt=-1), dict(group=16), dict(group=48), dict(group=0),
                dict(fmt=1, group=64), dict(M=-1), dict(N=0), dict(K=0), dict(K=240),
                dict(K=192, group=128), dict(act=2), dict(act=1, N=63), dict(out_dtype=3),
                dict(x=None), dict(codes=None), dict(scale=None), dict(out=None), dict(x=ODD),
                dict(codes=ODD), dict(scale=ODD), dict(out=ctypes.c_void_p(0x10001)),
                dict(add=ctypes.c_void_p(0x10001)),
                dict(out_dtype=1, out=ctypes.c_void_p(0x10002))):
        assert c(**bad) == INV, bad
    for big in (dict(M=(1 << 24) + 1), dict(N=(1 << 24) + 1), dict(K=1 << 23)):
        assert c(**big) == UNS, big
    assert c(M=0, x=None) == OK
    ws = ops.lib().qmoe_w4_matmul_workspace
    for bad in ((-1, 8, 256), (4, 0, 256), (4, 8, 0), (4, 8, 200)):
        assert ws(*bad) == 0
    for M, N, K in ((1, 64, 4096), (64, 64, 16384), (100, 256, 8192), (300, 128, 32768)):
        need = ws(M, N, K)
        assert need % 256 == 0
        if need:
            at = dict(M=M, N=N, K=K)
            assert c(**at, ws_bytes=need - 1) == INV and c(**at, ws=None) == INV
            assert c(**at, ws=ODD) == INV


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _al(T, k, E, bm=16):
    cap = ops.align_capacity(T, k, E, bm)
    i = torch.int32
    return {"sorted_pair_ids": _z(cap, dtype=i), "tile_expert": _z(cap // bm, dtype=i),
            "expert_offsets": _z(E + 1, dtype=i), "num_padded": _z(1, dtype=i), "block_m": bm}


F32, U8, F16, I32 = torch.float32, torch.uint8, torch.float16, torch.int32


@pytest.mark.parametrize("call", [
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(4, 2, 8), 2, act="gelu"),
    lambda: ops.grouped_matmul(_z(4, 64), _z(32, 64), _al(4, 2, 8), 2),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 72), _al(4, 2, 8), 2),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(4, 2, 8), 2, trans=True),
    lambda: ops.grouped_matmul(_z(4, 64, dtype=F32), _z(8, 32, 64), _al(4, 2, 8), 2),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64, dtype=F32), _al(4, 2, 8), 2),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(4, 2, 8), 2, out_dtype=F16),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(5, 2, 8), 2),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(4, 2, 9), 2),
    lambda: ops.grouped_matmul(_z(5, 64), _z(8, 32, 64), _al(4, 2, 8), 2, pair_rows=True),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(4, 2, 8), 2, gu=_z(8, 32)),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(4, 2, 8), 2, act="silu_mul",
                               gu=_z(8, 16)),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 64, 32), _al(4, 2, 8), 2, trans=True,
                               act="silu_mul"),
    lambda: ops.grouped_matmul(_z(8, 64), _z(8, 64, 32), _al(4, 2, 8), 2, pair_rows=True,
                               trans=True, act="silu_mul_backward"),
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(4, 2, 8), 2, out=_z(8, 33)),
    lambda: ops.grouped_wgrad(_z(8, 32), _z(5, 64), _al(4, 2, 8), 2),
    lambda: ops.grouped_wgrad(_z(8, 32, dtype=F32), _z(4, 64), _al(4, 2, 8), 2),
    lambda: ops.grouped_wgrad(_z(8, 32), _z(4, 64), _al(4, 2, 8), 2, accumulate=True),
    lambda: ops.grouped_wgrad(_z(8, 32), _z(4, 64), _al(4, 2, 8), 2, out=_z(8, 32, 64),
                              out_dtype=torch.bfloat16, accumulate=True),
    lambda: ops.grouped_wgrad(_z(8, 32), _z(4, 64), _al(4, 2, 8), 2, out=_z(8, 32, 65, dtype=F32)),
    lambda: ops.combine_backward(_z(4, 64), _z(8, 64, dtype=F32), _z(4, 2, dtype=I32),
                                 _z(4, 2, dtype=F32), 8),
    lambda: ops.combine_backward(_z(4, 64), _z(8, 64), _z(4, 2, dtype=torch.int64),
                                 _z(4, 2, dtype=F32), 8),
    lambda: ops.combine_backward(_z(4, 64), _z(8, 64), _z(4, 2, dtype=I32), _z(4, 2, dtype=F32), 8,
                                 add=_z(4, 9, dtype=F32)),
    lambda: ops.w4_matmul(_z(4, 64), _z(8, 32, dtype=U8), _z(8, 2, dtype=F16), act="gelu"),
    lambda: ops.w4_matmul(_z(4, 64, dtype=F16), _z(8, 32, dtype=U8), _z(8, 2, dtype=F16)),
    lambda: ops.w4_matmul(_z(4, 64), _z(8, 64, dtype=U8), _z(8, 2, dtype=F16)),
    lambda: ops.w4_matmul(_z(4, 64), _z(8, 32, dtype=U8), _z(8, 4, dtype=F16)),
    lambda: ops.w4_matmul(_z(4, 64), _z(8, 32, dtype=U8), _z(8, 1, dtype=U8)),
    lambda: ops.w4_matmul(_z(4, 64), _z(8, 32, dtype=U8), _z(8, 0, dtype=F16)),
    lambda: ops.w4_matmul(_z(4, 64), _z(8, 32, dtype=U8), _z(7, 2, dtype=F16)),
    lambda: ops.w4_matmul(_z(4, 64), _z(9, 32, dtype=U8), _z(9, 2, dtype=F16), act="silu_mul"),
    lambda: ops.w4_matmul(_z(4, 64), _z(8, 32, dtype=U8), _z(8, 2, dtype=F16), add=_z(4, 4)),
    # right shapes and types, but not on a GPU
    lambda: ops.grouped_matmul(_z(4, 64), _z(8, 32, 64), _al(4, 2, 8), 2),
    lambda: ops.grouped_wgrad(_z(8, 32), _z(4, 64), _al(4, 2, 8), 2),
    lambda: ops.combine_backward(_z(4, 64), _z(8, 64), _z(4, 2, dtype=I32), _z(4, 2, dtype=F32), 8),
    lambda: ops.w4_matmul(_z(4, 64), _z(8, 32, dtype=U8), _z(8, 2, dtype=F16)),
])
def test_binding_refusals(call):
    with pytest.raises(ValueError):
        call()
