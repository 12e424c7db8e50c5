"""The training entry points on the host: sizes whose launches would pass 2^32
threads along a grid's dimension are refused before anything is launched. No
GPU is needed."""
import ctypes

import mixture_experts_layer_count_amd as moe

INVALID, UNSUPPORTED, WS_SMALL = 1, 2, 3
F32, BF16 = 0, 1
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first


def test_checkpoint_values_past_a_launch():
    """A launch packs 4096 values with 256 threads: 2^36 values need 2^32."""
    pack, unpack = moe.lib().moe_checkpoint_pack, moe.lib().moe_checkpoint_unpack
    for R, C in ((1 << 16, 1 << 20), ((1 << 31) - 1, 64), (1 << 31, 32), (1 << 62, 32), ((1 << 36) // 96, 96)):
        for dt in (F32, BF16):
            assert pack(FAKE, dt, C, R, C, FAKE, FAKE, None) == UNSUPPORTED, (R, C)
            assert unpack(FAKE, FAKE, R, C, dt, FAKE, None) == UNSUPPORTED, (R, C)


def test_router_tokens_past_a_launch():
    """64 tokens take 256 threads at most: 2^30 tokens need 2^32."""
    loss, back = moe.lib().moe_balance_loss, moe.lib().moe_route_backward
    for T, E in (((1 << 30) - 63, 1), (1 << 30, 1), ((1 << 31) - 1, 1), ((1 << 30) - 1, 2)):
        assert loss(FAKE, FAKE, T, E, 1, None, 1, 0.1, 0.1, FAKE, FAKE, FAKE, FAKE, 1 << 50, None) == UNSUPPORTED, T
        assert back(FAKE, FAKE, FAKE, FAKE, T, E, 1, None, 1, FAKE, 0.1, 0.1, None, FAKE, None) == UNSUPPORTED, T
    # the workspace of sizes near the limit, formed in 64 bits
    ws = moe.lib().moe_balance_loss_workspace_bytes
    assert 0 < ws((1 << 30) - 1024, 1, 1) <= ws((1 << 30) - 64, 1, 1)
    assert ws((1 << 31) - 1, 1, 1) < 1 << 30  # partial rows of 64 tokens


def test_train_plan():
    """The tile heights and the down product of given sizes; refusals as the FFN calls'."""
    v = [ctypes.c_int(-1) for _ in range(3)]
    out = [ctypes.byref(x) for x in v]
    plan = moe.lib().moe_ffn_train_plan
    for sizes, want in (((4096, 2, 8, 4096, 14336), [256, 256, 0]), ((4096, 1, 32, 7168, 2048), [128, 128, 0]),
                        ((8192, 8, 128, 2048, 768), [256, 256, 1]), ((1536, 2, 8, 640, 416), [128, 128, 0]),
                        ((0, 1, 1, 32, 32), [128, 128, 0])):
        assert plan(*sizes, *out) == 0 and [x.value for x in v] == want, sizes
    assert plan(64, 65, 8, 256, 96, *out) == UNSUPPORTED and plan(64, 2, 8, 250, 96, *out) == UNSUPPORTED
    assert plan(-1, 2, 8, 256, 96, *out) == INVALID and plan(64, 0, 8, 256, 96, *out) == INVALID
    for i in range(3):
        assert plan(64, 2, 8, 256, 96, *(None if j == i else o for j, o in enumerate(out))) == INVALID


def test_balance_loss_workspace_alignment():
    """The workspace holds counters and fp32 sums: off the 4-byte boundary it is refused."""
    loss = moe.lib().moe_balance_loss
    for at in (0x1001, 0x1002, 0x1003):
        assert loss(FAKE, FAKE, 64, 8, 2, None, 1, 0.1, 0.1, FAKE, FAKE, FAKE, ctypes.c_void_p(at), 1 << 50,
                    None) == WS_SMALL
