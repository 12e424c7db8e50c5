"""GPU: what holds bit for bit around the 4-bit operators. A row of the W4A4 FFN is summed
in one order whatever tile or piece it lies in, so the layer is its stages exactly; and
quantising what was read back gives the codes again, where no value is subnormal."""
import pytest
import torch

import mixture_experts_layer_count_amd as moe
from _gpu import say
from test_gpu_mx4 import _ffn, _layer, _values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


# one row to several tiles of each height, by row and by token, with whole and part rounds
@pytest.mark.parametrize("T,H,F,E,k,Fs,shared", [(1, 256, 128, 8, 2, 0, None), (130, 384, 160, 8, 3, 160, "mxfp4"),
                                                 (700, 256, 416, 16, 4, 0, None), (2500, 512, 256, 4, 1, 256, "mxfp4"),
                                                 (3300, 1088, 64, 12, 5, 64, "mxfp4"), (600, 5888, 96, 4, 2, 96, "mxfp4")])
def test_layer_is_its_stages(T, H, F, E, k, Fs, shared):
    say(f"[mx4 exact] layer T={T} H={H} F={F} E={E} k={k} shared {shared}")
    d = _layer(T, H, F, E, k, Fs, shared, T)
    Y, _, idx, w, _ = moe.MoELayer(d, k, path="tiled_a4").forward(d["X"], aux=True)
    _, off, src, back, _ = moe.permute(idx, E)
    Yp = _ffn(d | {"offsets": off, "row_src": src, "k": k})
    S = None
    if Fs:
        one = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        S = moe.grouped_ffn(d["X"], one, *(d[n].unsqueeze(0) for n in ("Ws1", "Ws3", "Ws2", "Ss1", "Ss3", "Ss2")),
                            path="tiled_a4")
    assert torch.equal(Y, moe.combine(Yp, back, w, S))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_codes_again(dt):
    say(f"[mx4 exact] quantised, read back to {dt}, quantised")
    x = _values(300, 2016, torch.float32, 5).cuda()
    Q, S = moe.quantize_mxfp4_rows(x)
    q, s = moe.quantize_mxfp4_rows(moe.dequantize_mxfp4_rows(Q, S, dt))
    keep = S >= 2                       # half of 2^-125 is the smallest normal number
    assert int(keep.sum()) > 18000 and int((S == 255).sum()) == 3 and int((S == 127).sum()) > 0
    assert torch.equal(s[keep], S[keep])
    groups = lambda t: t.view(300, 63, 16)[keep]  # noqa: E731
    assert torch.equal(groups(q), groups(Q))
    w = x.view(5, 60, 2016)[:, :32].contiguous()
    Q, S = moe.quantize_mxfp4_weights(w)
    q, s = moe.quantize_mxfp4_weights(moe.dequantize_mxfp4_weights(Q, S, dt))
    keep = S >= 2
    cols = keep.expand(5, 16, 2016)
    assert torch.equal(s[keep], S[keep]) and torch.equal(q[cols], Q[cols])
