"""The W4A4 path on the host: workspaces and sizes that its launches cannot take are
answered with a status before anything is launched. No GPU is needed."""
import ctypes

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
