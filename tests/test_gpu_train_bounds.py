"""GPU: the training operators on the bounds-checked build (libmoe_debug.so).

A row number that the kernels would address memory with, planted out of range,
sets its bit and is taken as 0; everything stays in bounds."""
import pytest
import torch

import mixture_experts_layer_count_amd as moe
from mixture_experts_layer_count_amd import _lib
from _gpu import say
import test_gpu_train_tall as tall
from test_gpu_train import _backward, _dev, _ffn_case, _forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()
    return _lib.load(_lib.DEBUG_LIB_PATH)


# -1 stays below 0 only before the division by k: as a token it would be 0
@pytest.mark.parametrize("bad", ["-1", "-k", "T*k"])
def test_debug_build_catches_row_src(debug_lib, bad):
    say(f"[train bounds] planted row_src {bad}")
    T, k = 40, 3
    c = _ffn_case(T, 64, 96, 4, k)
    d = _dev(c)
    _, ck = _forward(d)
    r = 17
    planted, zero = dict(d), dict(d)
    planted["row_src"], zero["row_src"] = d["row_src"].clone(), d["row_src"].clone()
    planted["row_src"][r] = {"-1": -1, "-k": -k, "T*k": T * k}[bad]
    zero["row_src"][r] = 0
    ref = (*_forward(zero)[0:1], *_backward(zero, ck))
    torch.cuda.synchronize()
    with _lib.use_library(debug_lib):
        debug_lib.moe_debug_bounds()
        Yp, _ = _forward(planted)
        assert debug_lib.moe_debug_bounds() == _lib.MOE_BOUNDS_A_ROW
        dX, dw, *dW = _backward(planted, ck)
        assert debug_lib.moe_debug_bounds() == _lib.MOE_BOUNDS_A_ROW
        # one product at a time: the routing weight's row, and the weight gradients' rows
        _backward(planted, ck, need=("dtopk_w",))
        assert debug_lib.moe_debug_bounds() == _lib.MOE_BOUNDS_A_ROW
    for a, b in zip((Yp, dX, dw, *dW), ref):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,H,F,E,k,skew,kernels", [
    (17000, 544, 608, 7, 2, 0.8, (256, 256, False)),
    (16500, 512, 320, 4, 2, 0.3, (256, 256, True)),
    (33000, 288, 4128, 3, 1, 0.1, (256, 256, False)),   # split last rounds of DOWN and DX
    (200, 4128, 64, 2, 1, 0.1, (128, 128, False)),      # and of 128-row GATE_UP and BACK
    (9000, 64, 96, 2, 1, 0.2, (128, 128, False)),       # experts of more rows than one window of row numbers
])
def test_debug_build_tall_and_split(debug_lib, T, H, F, E, k, skew, kernels):
    say(f"[train bounds] ffn T={T} H={H} F={F} E={E} k={k}")
    assert tall.plan(T, H, F, E, k) == kernels
    d = tall._case(T, H, F, E, k, skew)
    Yp, ck = tall._forward(d)
    got = tall._backward(d, ck)
    torch.cuda.synchronize()
    with _lib.use_library(debug_lib):
        debug_lib.moe_debug_bounds()
        Yd, cd = tall._forward(d)
        gd = tall._backward(d, cd)
        assert debug_lib.moe_debug_bounds() == 0
    for a, b in zip((Yp, *ck, *got), (Yd, *cd, *gd)):
        assert torch.equal(a, b)
