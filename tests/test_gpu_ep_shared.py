"""GPU: expert-parallel ranks whose shared expert is bf16 beside experts on a quantised
path (W4A4, W8A8): the layer takes such weights, and runs the shared expert on the bf16
tiled kernels."""
import pytest
import torch

import mixture_experts_layer_count_amd as moe
import oracle
from synth import MINI_CONFIGS
from _gpu import rel_err, say, screened_layer, tol_for
from test_gpu_mx4 import _ffn, _layer

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and bf16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def _composed(d, k, G, path):
    """The ranks' result, and the same by their returned rows and the shared expert's call."""
    X = d["X"]
    T = X.shape[0]
    epl = moe.EPLoopback(d, k, G, path=path)
    Y = epl.forward(X, keep=True)
    st = epl.last
    one = [d[n].unsqueeze(0) for n in ("Ws1", "Ws3", "Ws2")]
    want, S = torch.empty_like(Y), torch.empty_like(Y)
    for r in range(G):
        sl = moe.rank_tokens(T, G, r)
        n = sl.stop - sl.start
        S[sl] = moe.grouped_ffn(X[sl], torch.tensor([0, n], dtype=torch.int32, device="cuda"), *one, path="tiled")
        want[sl] = moe.combine(st["ret"][r, :n * k], st["send_slot"][r, :n * k], st["routes"][r][2], S[sl])
    return Y, want, S


@pytest.mark.parametrize("G", [1, 4])
def test_w4a4_ranks(G):
    T, H, F, E, k, Fs = 161, 256, 128, 16, 3, 96
    say(f"[ep] W4A4 and a bf16 shared expert, {G} ranks")
    d = _layer(T, H, F, E, k, Fs, "bf16", 7)
    X = d["X"]
    Y, want, S = _composed(d, k, G, "tiled_a4")
    assert torch.equal(Y, want)
    # the layer on one rank: its logits are the same fp32 sums (H U of their terms) in another
    # split, which moves a weight by twice that; S, its h and Y may round to bf16 the other way
    L, logits, idx, w, _ = moe.MoELayer(d, k, path="tiled_a4").forward(X, aux=True)
    _, off, src, back, _ = moe.permute(idx, E)
    Yp = _ffn(d | {"offsets": off, "row_src": src, "k": k}).float()[back.long()].view(T, k, H).abs()
    dz = H * U * (X.float().abs() @ d["Wg"].float().abs()).max()
    h = torch.nn.functional.silu(X.float() @ d["Ws1"].float()) * (X.float() @ d["Ws3"].float())
    dS = 2 * HALF * (1.01 * (h.abs() @ d["Ws2"].float().abs()) + S.float().abs())
    tol = dS + 2 * (2 * dz + (k + 2) * U) * (w.unsqueeze(2) * Yp).sum(1)
    assert ((Y.float() - L.float()).abs() <= tol + 2 * HALF * (L.float().abs() + tol)).all()


@pytest.mark.parametrize("name,G", [("mini_fp8_bf16s_decode", 2), ("mini_fp8_bf16s_prefill", 4)])
def test_w8a8_ranks(name, G):
    cfg = MINI_CONFIGS[name]
    say(f"[ep] W8A8, {name}, {G} ranks")
    d = screened_layer(cfg)
    Y, want, _ = _composed(d, cfg.k, G, "tiled_a8")
    assert torch.equal(Y, want)
    ref = oracle.forward_tokens(oracle.Layer(d, cfg.k), range(cfg.T))["Y"]
    assert rel_err(Y, ref) <= tol_for(cfg)
