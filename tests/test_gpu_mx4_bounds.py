"""GPU: the W4A4 expert FFN on the bounds-checked build (libmoe_debug.so).

A gathered row planted below 0 sets its bit and is taken as assignment 0, in each of the
kernels that quantise the rows; nothing is read out of bounds. (The token rows' number is
not known to moe_grouped_ffn, so entries past them cannot be told.)"""
import pytest
import torch

import mixture_experts_layer_count_amd as moe
from mixture_experts_layer_count_amd import _lib
from _gpu import say
from test_gpu_mx4 import _case, _ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()
    return _lib.load(_lib.DEBUG_LIB_PATH)


# a row a thread, four rows a thread, token by token (few rows and many, 2 and 4 picks). -1
# stays below 0 only before the division by k: as a token it would be 0
@pytest.mark.parametrize("bad", ["-1", "-k", "lowest"])
@pytest.mark.parametrize("T,H,F,E,k", [(40, 64, 96, 4, 2), (9000, 1056, 64, 4, 2), (16000, 1056, 64, 6, 4)])
def test_debug_build_catches_row_src(debug_lib, T, H, F, E, k, bad):
    say(f"[mx4 bounds] planted row_src {bad}, T={T} k={k}")
    d = _case(T, H, F, E, k, T)
    planted, zero = d["row_src"].clone(), d["row_src"].clone()
    for r in (17, T * k - 1):
        planted[r] = {"-1": -1, "-k": -k, "lowest": -2 ** 31}[bad]
        zero[r] = 0
    ref = _ffn(d | {"row_src": zero})
    torch.cuda.synchronize()
    with _lib.use_library(debug_lib):
        debug_lib.moe_debug_bounds()
        Y = _ffn(d | {"row_src": planted})
        assert debug_lib.moe_debug_bounds() == _lib.MOE_BOUNDS_A_ROW
        # and nothing where all rows are in range
        assert torch.equal(_ffn(d | {"row_src": zero}), ref) and debug_lib.moe_debug_bounds() == 0
    assert torch.equal(Y, ref)
