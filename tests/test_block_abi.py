"""The operators around the experts without a GPU: every bad argument of the
C ABI and of the binding is refused before anything is launched."""
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
NAN, INF = float("nan"), float("inf")


def _caller(name, **base):
    """A call of `name` with the arguments `base` (in order), some replaced."""
    fn = getattr(ops.lib(), name)

    def call(**kw):
        assert set(kw) <= set(base)
        return fn(*{**base, **kw}.values())
    return call


def test_fp8_quant_refusals():
    c = _caller("qmoe_fp8_quant", x=P, dtype=0, B=1, M=4, K=256, block=0, act=0, codes=P, scale=P,
                codes_t=P, scale_t=P, stream=None)
    for bad in (dict(dtype=2), dict(B=-1), dict(M=-1), dict(K=0), dict(block=2), dict(act=2),
                dict(B=2), dict(block=1, act=1), dict(x=None), dict(scale=None),
                dict(codes=None), dict(scale_t=None), dict(codes_t=None),
                dict(codes=None, scale=None, codes_t=None, scale_t=None), dict(codes=ODD),
                dict(codes_t=ODD), dict(x=ctypes.c_void_p(0x10001)),
                dict(scale=ctypes.c_void_p(0x10002))):
        assert c(**bad) == INV, bad
    assert c(block=1, B=70000) == UNS
    assert c(M=65535 * 128 + 1) == UNS and c(K=(1 << 29) + 1) == UNS
    assert c(M=0, x=None) == OK and c(B=0, x=None) == OK


def test_fp8_matmul_refusals():
    c = _caller("qmoe_fp8_matmul", a=P, a_scale=P, b=P, b_scale=P, b_block=1, M=4, N=8, K=256,
                out=P, out_dtype=0, ws=P, ws_bytes=1 << 40, stream=None)
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=200), dict(b_block=2), dict(out_dtype=2),
                dict(a=None), dict(a_scale=None), dict(b=None), dict(b_scale=None),
                dict(out=None), dict(a=ODD), dict(b=ODD), dict(out=ctypes.c_void_p(0x10001)),
                dict(out=ctypes.c_void_p(0x10002), out_dtype=1)):
        assert c(**bad) == INV, bad
    for big in (dict(M=(1 << 24) + 1), dict(N=(1 << 24) + 1), dict(K=1 << 25)):
        assert c(**big) == UNS, big
    assert c(M=0, a=None) == OK
    ws = ops.lib().qmoe_fp8_matmul_workspace
    for bad in ((-1, 8, 256), (4, 0, 256), (4, 8, 0), (4, 8, 200)):
        assert ws(*bad) == 0
    for M, N, K in ((1, 64, 4096), (64, 64, 16384), (300, 128, 8192), (512, 512, 32768)):
        need = ws(M, N, K)
        assert need % 256 == 0
        if need:  # a split product refuses a short, missing or misaligned workspace
            assert c(M=M, N=N, K=K, ws_bytes=need - 1) == INV
            assert c(M=M, N=N, K=K, ws=None) == INV
            assert c(M=M, N=N, K=K, ws=ODD) == INV


def test_fp8_grouped_matmul_refusals():
    c = _caller("qmoe_fp8_grouped_matmul", a=P, a_scale=P, pair_rows=0, b=P, b_scale=P, srt=P,
                te=P, off=P, npad=P, T=4, k=2, E=8, block_m=16, N=64, K=256, out=P, out_dtype=0,
                stream=None)
    for bad in (dict(pair_rows=2), dict(T=-1), dict(k=0), dict(k=9), dict(E=0), dict(block_m=48),
                dict(N=0), dict(K=64), dict(K=0), dict(out_dtype=5), dict(T=1 << 30), dict(a=None),
                dict(a_scale=None), dict(b=None), dict(b_scale=None), dict(srt=None),
                dict(te=None), dict(off=None), dict(npad=None), dict(out=None),
                dict(a=ODD), dict(b=ODD)):
        assert c(**bad) == INV, bad
    assert c(E=2000) == UNS
    assert c(T=0, a=None) == OK


def test_balance_refusals():
    ws = ops.lib().qmoe_balance_workspace
    n = ws(6400, 8)
    assert n >= 256 and n % 256 == 0 and ws(-1, 8) == 0 and ws(4, 0) == 0
    c = _caller("qmoe_balance", logits=P, ids=P, mask=None, T=6400, E=8, k=2, coef=0.1, loss=P,
                counts=P, probs=P, tokens=P, ws=P, ws_bytes=n, stream=None)
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(E=64, k=17),
                dict(T=(1 << 29) + 1), dict(coef=NAN),
                dict(coef=INF), dict(logits=None), dict(ids=None), dict(loss=None),
                dict(counts=None), dict(probs=None), dict(tokens=None), dict(ws=None),
                dict(ws_bytes=n - 1), dict(ws=ODD)):
        assert c(**bad) == INV, bad
    assert c(E=1025, ws_bytes=1 << 40) == UNS
    b = _caller("qmoe_balance_backward", logits=P, mask=None, counts=P, tokens=P, dloss=P, T=64,
                E=8, k=2, coef=0.1, dlogits=P, stream=None)
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(T=(1 << 29) + 1), dict(coef=INF),
                dict(logits=None), dict(counts=None), dict(tokens=None),
                dict(dloss=None), dict(dlogits=None)):
        assert b(**bad) == INV, bad
    assert b(E=1025) == UNS
    assert b(T=0, logits=None) == OK


def test_norm_refusals():
    pre = _caller("qmoe_pre_norm", x=P, dtype=0, w=P, eps=1e-6, T=4, H=64, form=3, n=P, scale=P,
                  stream=None)
    post = _caller("qmoe_post_norm", y=P, x=P, dtype=0, w=P, gate=P, kind=1, alpha=1.0, eps=1e-6,
                   T=4, H=64, out=P, next_w=P, form=2, n=P, scale=P, stream=None)
    n = ops.lib().qmoe_norm_backward_workspace(64)
    assert n > 0 and n % 256 == 0
    assert ops.lib().qmoe_norm_backward_workspace(0) == 0
    assert ops.lib().qmoe_norm_backward_workspace(16392) == 0
    preb = _caller("qmoe_pre_norm_backward", dn=P, x=P, dtype=0, w=P, eps=1e-6, dres=None, T=4,
                   H=64, dx=P, dw=P, ws=P, ws_bytes=n, stream=None)
    postb = _caller("qmoe_post_norm_backward", dout=P, y=P, dtype=0, w=P, gate=P, kind=3,
                    alpha=1.0, eps=1e-6, T=4, H=64, dy=P, dres=P, dw=P, dgate=P, ws=P, ws_bytes=n,
                    stream=None)
    for c in (pre, post, preb, postb):
        big = {} if c in (pre, post) else {"ws_bytes": 1 << 40}
        for bad in (dict(dtype=2), dict(T=-1), dict(H=0), dict(eps=0.0), dict(eps=-1.0),
                    dict(eps=NAN), dict(eps=INF)):
            assert c(**bad) == INV, bad
        assert c(H=16392, **big) == UNS
        assert c(H=8193, **big) == UNS            # no 16-byte loads above 8192 columns
        assert c(H=8200, w=ODD, **big) == UNS
    for bad in (dict(form=5), dict(form=-1), dict(x=None), dict(w=None), dict(n=None),
                dict(scale=None)):
        assert pre(**bad) == INV, bad
    for bad in (dict(kind=4), dict(kind=-1), dict(alpha=NAN), dict(form=7), dict(y=None),
                dict(x=None), dict(w=None), dict(gate=None), dict(out=None), dict(n=None),
                dict(scale=None)):
        assert post(**bad) == INV, bad
    assert pre(T=0, x=None) == OK and post(T=0, y=None) == OK
    for bad in (dict(dn=None), dict(x=None), dict(w=None), dict(dx=None), dict(dw=None),
                dict(ws=None), dict(ws_bytes=n - 1), dict(ws=ODD)):
        assert preb(**bad) == INV, bad
    for bad in (dict(dout=None), dict(y=None), dict(w=None), dict(gate=None), dict(dy=None),
                dict(dres=None), dict(dw=None), dict(dgate=None), dict(ws=None), dict(kind=9),
                dict(alpha=INF), dict(ws_bytes=n - 1), dict(ws=ODD)):
        assert postb(**bad) == INV, bad


def _z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


U8, BF = torch.uint8, torch.bfloat16


@pytest.mark.parametrize("call", [
    lambda: ops.fp8_quant(_z(4, 128), act="gelu"),
    lambda: ops.fp8_quant(_z(4, 128), rows=False),
    lambda: ops.fp8_quant(_z(4, 128), block=True, act="silu_mul"),
    lambda: ops.fp8_quant(_z(2, 4, 128)),
    lambda: ops.fp8_quant(_z(4, 128, dtype=torch.float16)),
    lambda: ops.fp8_matmul(_z(4, 200, dtype=U8), _z(1, 4), _z(8, 200, dtype=U8), _z(1, 1)),
    lambda: ops.fp8_matmul(_z(4, 256, dtype=U8), _z(4, 2), _z(8, 256, dtype=U8), _z(1, 2)),
    lambda: ops.fp8_matmul(_z(4, 256, dtype=U8), _z(2, 4), _z(8, 256, dtype=U8), _z(2, 8)),
    lambda: ops.fp8_matmul(_z(4, 256, dtype=U8), _z(2, 4), _z(8, 128, dtype=U8), _z(1, 1)),
    lambda: ops.fp8_matmul(_z(4, 256), _z(2, 4), _z(8, 256, dtype=U8), _z(1, 2)),
    lambda: ops.fp8_matmul(_z(4, 256, dtype=U8), _z(2, 4), _z(8, 256, dtype=U8), _z(1, 2),
                           out_dtype=torch.float16),
    lambda: ops.balance_loss(_z(4, 8), _z(3, 2, dtype=torch.int32)),
    lambda: ops.balance_loss(_z(4, 8), _z(4, 2, dtype=torch.int64)),
    lambda: ops.balance_loss(_z(4, 8, dtype=BF), _z(4, 2, dtype=torch.int32)),
    lambda: ops.balance_loss_backward(_z(4, 8), _z(8), _z(1, dtype=torch.int32), 2, _z(1)),
    lambda: ops.pre_norm(_z(4, 8), _z(9)),
    lambda: ops.pre_norm(_z(4, 8), _z(8, dtype=BF)),
    lambda: ops.pre_norm(_z(4, 8, dtype=torch.float16), _z(8)),
    lambda: ops.post_norm(_z(4, 8), _z(8), _z(4, 8, dtype=BF)),
    lambda: ops.post_norm_backward(_z(4, 8), _z(4, 9), _z(9)),
    lambda: ops.pre_norm_backward(_z(4, 8), _z(4, 8), _z(8), dres=_z(3, 8)),
    # right shapes and types, but not on a GPU
    lambda: ops.fp8_quant(_z(4, 128)),
    lambda: ops.fp8_matmul(_z(4, 256, dtype=U8), _z(2, 4), _z(8, 256, dtype=U8), _z(1, 2)),
    lambda: ops.balance_loss(_z(4, 8), _z(4, 2, dtype=torch.int32)),
    lambda: ops.pre_norm(_z(4, 8), _z(8)),
    lambda: ops.post_norm(_z(4, 8), _z(8), _z(4, 8)),
])
def test_binding_refusals(call):
    with pytest.raises(ValueError):
        call()
