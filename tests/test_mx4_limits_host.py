"""The W4A4 path on the host: workspaces and sizes that its launches cannot take are
answered with a status before anything is launched. No GPU is needed."""
import ctypes

import pytest
import torch

import mixture_experts_layer_count_amd as moe
from test_abi_host import _desc, _ffn
from test_mx4_host import A4, FAKE, MX, WS_SMALL


def _forward(ws=FAKE, T=100, **kw):
    d = dict(H=512, F=1024, w_dt=3, S1=0x1000, S3=0x1000, S2=0x1000, path=A4) | kw
    return moe.lib().moe_forward(ctypes.byref(_desc(**d)), FAKE, T, FAKE, ws, 1 << 62, None, None, None, None, None, None)


def test_workspace_alignment():
    """The panels in it are copied and stored 16 bytes at a time."""
    for at in (0x1001, 0x1004, 0x1008):
        ws = ctypes.c_void_p(at)
        assert _ffn(moe.lib(), ws=ws, ws_bytes=1 << 60, path=A4, **MX) == WS_SMALL
        assert _forward(ws) == WS_SMALL


def test_sizes_past_a_launch():
    """64 rows of a panel take 256 to 1024 threads, a workgroup of 512 up to 64 tiles: sizes
    that need 2^32 threads are refused, and have no workspace."""
    lib = moe.lib()
    size = lambda M, G, H, F: lib.moe_grouped_ffn_workspace_bytes(M, G, H, F, 1, 3, A4)  # noqa: E731
    at_most = 4194302                                   # blocks of 256 rows and a panel, beside the tile list's
    for M, G, H, F in ((1 << 30, 1, 32, 32), (256 * at_most + 1, 8, 128, 64), (128 * at_most + 1, 8, 160, 64),
                       (1 << 20, 4, 1 << 20, 32),       # rows
                       (64, 1 << 30, 32, 32), (64, 1 << 21, 32, 1 << 20), (64, 1 << 21, 1 << 20, 32)):  # tiles
        assert size(M, G, H, F) == 0, (M, G, H, F)
        assert _ffn(lib, M=M, G=G, H=H, F=F, ws_bytes=(1 << 63), path=A4, **MX) == 2, (M, G, H, F)
    # up to there the size is what counts
    for M, G, H, F in ((256 * at_most, 8, 128, 64), (128 * at_most - 256, 8, 160, 64), (64, 1 << 25, 32, 32)):
        assert 0 < size(M, G, H, F) < 1 << 62
        assert _ffn(lib, M=M, G=G, H=H, F=F, ws_bytes=64, path=A4, **MX) == WS_SMALL, (M, G, H, F)
    # the layer: 65535 tokens of the widest rows
    big = dict(H=1 << 20, E=64, k=64)
    d = _desc(F=1024, w_dt=3, S1=0x1000, S3=0x1000, S2=0x1000, path=A4, **big)
    assert lib.moe_forward_workspace_bytes(ctypes.byref(d), 65535) == 0 < lib.moe_forward_workspace_bytes(ctypes.byref(d), 500)
    assert _forward(T=65535, **big) == 2


class _Tensor:
    """What the binding asks of a device tensor, on a machine without one."""
    is_cuda = True

    def __init__(self, shape, dtype, device="cuda:0"):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 0x1000


@pytest.mark.parametrize("name", ["offsets", "W1", "S2", "row_src", "out"])
def test_operands_on_another_device(name):
    """A call runs on its rows' device; whatever lies elsewhere is refused by name."""
    G, H, F, T, k = 4, 64, 96, 5, 2
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    a = {"Xin": ((T, H), bf), "offsets": ((G + 1,), i32), "W1": ((G, H // 2, F), u8), "W3": ((G, H // 2, F), u8),
         "W2": ((G, F // 2, H), u8), "S1": ((G, H // 32, F), u8), "S3": ((G, H // 32, F), u8),
         "S2": ((G, F // 32, H), u8), "row_src": ((T * k,), i32), "out": ((T * k, H), bf)}
    t = {n: _Tensor(*v) for n, v in a.items()}
    t[name] = _Tensor(*a[name], device="cuda:1")
    with pytest.raises(ValueError, match=name):
        moe.grouped_ffn(**t, k=k, path="tiled_a4")
