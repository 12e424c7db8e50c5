"""The 4-bit and the dispatch-gradient entry points on the host: arguments are
answered with status codes before anything is launched, and the binding refuses
tensors the calls cannot take. No GPU is needed."""
import ctypes

import pytest
import torch

import mixture_experts_layer_count_amd as moe
from mixture_experts_layer_count_amd import _lib
from test_abi_host import _desc, _ffn

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
F32, BF16, FP8, MXFP4 = 0, 1, 2, 3
A4 = _lib.PATHS["tiled_a4"]
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1004)   # on no 8- or 16-byte boundary
HALF = ctypes.c_void_p(0x1008)  # on an 8-byte boundary
MX = dict(w_dt=MXFP4, S1=FAKE, S3=FAKE, S2=FAKE)


def test_rows_validation():
    lib = moe.lib()
    q = lambda X=FAKE, dt=BF16, ldx=64, R=4, C=64, Q=FAKE, S=FAKE: lib.moe_quantize_mxfp4_rows(X, dt, ldx, R, C, Q, S, None)  # noqa: E731
    d = lambda Q=FAKE, S=FAKE, R=4, C=64, dt=BF16, Y=FAKE: lib.moe_dequantize_mxfp4_rows(Q, S, R, C, dt, Y, None)  # noqa: E731
    assert q(None, R=0, Q=None, S=None) == OK and d(None, None, R=0, Y=None) == OK
    assert q(R=-1) == INVALID and q(C=0) == INVALID and q(ldx=32) == INVALID
    assert q(None) == INVALID and q(Q=None) == INVALID and q(S=None) == INVALID
    assert q(dt=FP8) == UNSUPPORTED and q(C=48, ldx=48) == UNSUPPORTED and q(ldx=68) == UNSUPPORTED
    assert q(dt=F32, ldx=66) == UNSUPPORTED and q(C=1 << 21, ldx=1 << 21) == UNSUPPORTED
    assert q(R=1 << 32) == UNSUPPORTED and d(R=1 << 32) == UNSUPPORTED
    assert q(HALF) == UNSUPPORTED and q(Q=ODD) == UNSUPPORTED and d(Q=ODD) == UNSUPPORTED and d(Y=HALF) == UNSUPPORTED
    assert d(dt=FP8) == UNSUPPORTED and d(None) == INVALID and d(S=None) == INVALID and d(Y=None) == INVALID


def test_weights_validation():
    lib = moe.lib()
    for f, n in ((lib.moe_quantize_mxfp4_weights, "q"), (lib.moe_dequantize_mxfp4_weights, "d")):
        def call(G=2, K=64, N=40, dt=BF16, W=FAKE, Q=FAKE, S=FAKE):
            return f(W, dt, G, K, N, Q, S, None) if n == "q" else f(Q, S, G, K, N, dt, W, None)
        assert call(G=0, W=None, Q=None, S=None) == OK
        assert call(G=-1) == INVALID and call(K=0) == INVALID and call(N=0) == INVALID
        assert call(W=None) == INVALID and call(Q=None) == INVALID and call(S=None) == INVALID
        assert call(dt=FP8) == UNSUPPORTED and call(K=48) == UNSUPPORTED and call(N=44) == UNSUPPORTED
        assert call(K=1 << 21) == UNSUPPORTED and call(G=1 << 20, K=1 << 10, N=1 << 10) == UNSUPPORTED
        assert call(W=HALF) == UNSUPPORTED and call(Q=ODD) == UNSUPPORTED and call(S=ODD) == UNSUPPORTED


def test_a4_path_validation():
    lib = moe.lib()
    ws = lib.moe_grouped_ffn_workspace_bytes
    # for MXFP4 experts alone, with their scales and bf16 tokens
    assert _ffn(lib, path=A4) == UNSUPPORTED
    assert _ffn(lib, path=A4, w_dt=FP8, S1=FAKE, S3=FAKE, S2=FAKE) == UNSUPPORTED
    assert _ffn(lib, path=A4, act_dt=F32, **MX) == UNSUPPORTED
    assert _ffn(lib, path=A4, **MX | dict(S2=None)) == INVALID
    assert _ffn(lib, path=A4, H=272, **MX) == UNSUPPORTED
    assert _ffn(lib, path=A4, M=0, Xin=None, **MX) == OK
    need = ws(64, 8, 256, 512, BF16, MXFP4, A4)
    assert need > 0 and _ffn(lib, path=A4, ws_bytes=need - 1, **MX) == WS_SMALL
    assert _ffn(lib, path=A4, ws=None, ws_bytes=1 << 40, **MX) == WS_SMALL
    # panels of codes and scale words: no bf16 h, and nothing that grows with the experts
    m, g, h, f = 65536, 8, 4096, 14336
    assert ws(m, g, h, f, BF16, MXFP4, A4) < ws(m, g, h, f, BF16, MXFP4, 2)
    # 4 is no path, and AUTO's choice for MXFP4 experts is as it was
    assert _ffn(lib, path=4, **MX) == INVALID
    assert ws(m, g, h, f, BF16, MXFP4, 0) == ws(m, g, h, f, BF16, MXFP4, 2)


def test_a4_alignment_and_limits():
    lib = moe.lib()
    big = dict(ws_bytes=1 << 60, path=A4, **MX)
    for n in ("Xin", "W1", "W3", "W2", "Yp"):
        assert _ffn(lib, **big | {n: HALF}) == UNSUPPORTED
    for n in ("S1", "S3", "S2"):
        assert _ffn(lib, **big | {n: ctypes.c_void_p(0x1002)}) == UNSUPPORTED
    assert _ffn(lib, **big | dict(M=(1 << 30) + 1)) == UNSUPPORTED
    d = dict(H=512, F=1024, w_dt=MXFP4, S1=0x1000, S3=0x1000, S2=0x1000, path=A4)
    forward = lambda X=FAKE, **kw: lib.moe_forward(  # noqa: E731
        ctypes.byref(_desc(**d | kw)), X, 100, FAKE, None, 0, None, None, None, None, None, None)
    assert forward() == WS_SMALL
    assert forward(HALF) == UNSUPPORTED and forward(W1=0x1008) == UNSUPPORTED and forward(S2=0x1001) == UNSUPPORTED
    assert lib.moe_quantize_mxfp4_rows(FAKE, BF16, 1 << 62, 1 << 62, 64, FAKE, FAKE, None) == UNSUPPORTED


def test_a4_layer_validation():
    ws = moe.lib().moe_forward_workspace_bytes
    mx = dict(H=512, F=1024, w_dt=MXFP4, S1=0x1000, S3=0x1000, S2=0x1000, path=A4)
    shared = dict(Ws1=0x1000, Ws3=0x1000, Ws2=0x1000)
    scales = dict(Ss1=0x1000, Ss3=0x1000, Ss2=0x1000)
    size = lambda T=100, **kw: ws(ctypes.byref(_desc(**mx | kw)), T)  # noqa: E731
    assert size() > 0
    assert size(Fs=1024, ws_dt=MXFP4, **shared, **scales) > size()
    assert size(Fs=512, ws_dt=MXFP4, **shared, **scales) == 0       # a width of its own
    assert size(Fs=96, ws_dt=BF16, **shared) > 0                    # beside it, in bf16
    assert size(w_dt=BF16, S1=None, S3=None, S2=None) == 0
    assert size(T=65536) == 0


def _combine(**kw):
    a = dict(dY=FAKE, Yp=FAKE, assign=FAKE, w=FAKE, n=None, T=8, k=2, H=64, dt=BF16, dYp=FAKE, dw=FAKE, stream=None) | kw
    return moe.lib().moe_combine_backward(*a.values())


def _permute(**kw):
    a = dict(dXp=FAKE, assign=FAKE, n=None, T=8, k=2, H=64, dt=BF16, add=None, dX=FAKE, stream=None) | kw
    return moe.lib().moe_permute_backward(*a.values())


def test_dispatch_gradient_validation():
    for f in (_combine, _permute):
        assert f(T=0) == OK
        for bad in (dict(T=-1), dict(k=0), dict(H=0), dict(assign=None)):
            assert f(**bad) == INVALID, bad
        for bad in (dict(dt=FP8), dict(H=62), dict(H=1 << 21), dict(k=65), dict(T=1 << 24), dict(T=1 << 23, k=64, H=1 << 19)):
            assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(dYp=None, dw=None), dict(dY=None), dict(Yp=None), dict(w=None)):
        assert _combine(**bad) == INVALID, bad
    for bad in (dict(dXp=None), dict(dX=None)):
        assert _permute(**bad) == INVALID, bad
    # 16 bytes, or 8 where a bf16 row is a multiple of 8 bytes alone
    assert _combine(dY=HALF) == UNSUPPORTED and _combine(Yp=HALF) == UNSUPPORTED and _combine(dYp=HALF) == UNSUPPORTED
    assert _permute(dXp=HALF) == UNSUPPORTED and _permute(add=HALF) == UNSUPPORTED and _permute(dX=HALF) == UNSUPPORTED
    assert _combine(dY=HALF, dt=F32, H=60) == UNSUPPORTED and _combine(dY=ODD, H=60) == UNSUPPORTED


def test_binding_refuses():
    x, i = torch.zeros(4, 64), torch.zeros(8, dtype=torch.int32)
    for call in (lambda: moe.quantize_mxfp4_rows(x), lambda: moe.quantize_mxfp4_weights(x),
                 lambda: moe.dequantize_mxfp4_rows(x.byte(), x.byte()[:, :4]),
                 lambda: moe.dequantize_mxfp4_weights(x.byte(), x.byte()[:4]),
                 lambda: moe.combine_backward(x, x.repeat(2, 1), i, torch.zeros(4, 2)),
                 lambda: moe.permute_backward(x, i[:4], 2)):
        with pytest.raises(ValueError):
            call()                                     # not on a device
    with pytest.raises(TypeError):
        moe.dequantize_mxfp4_rows(x, x)
    with pytest.raises(ValueError):
        moe.quantize_mxfp4_weights(x[0])               # neither [K,N] nor [G,K,N]
    with pytest.raises(ValueError):
        moe.permute_backward(x, i[:4], 3)              # 4 rows are no T * 3
    with pytest.raises(TypeError):
        moe.combine_backward(x.half(), x.half(), i, torch.zeros(4, 2))
