"""GPU: the training operators at the largest launches their sizes allow.

A launch holds fewer than 2^32 threads along each dimension of its grid; the
calls take sizes beyond what one dimension can count."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_count_amd as moe
from _gpu import say
from test_gpu_train import _check_backward, _check_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()
    yield
    torch.cuda.empty_cache()


def _dense(T, H, F, seed):
    """One expert over T tokens in row order, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    return {"X": bf(T, H), "W1": bf(1, H, F).mul_(0.2), "W3": bf(1, H, F).mul_(0.2), "W2": bf(1, F, H).mul_(0.2),
            "offsets": torch.tensor([0, T], dtype=torch.int32, device="cuda")}


def test_ffn_train_tokens_times_a_block_past_32_bits():
    """T * 256 threads do not fit 32 bits. Only the last tokens have a gradient,
    so the weight gradients are theirs alone."""
    T, H, F, n = (1 << 24) + 40, 32, 32, 60
    say(f"[limits] ffn T={T} H={H} F={F}")
    d = _dense(T, H, F, 1)
    last = slice(T - n, T)
    dY = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    dY[last] = torch.randn(n, H, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    Yp, ck = moe.ffn_train_forward(d["X"], d["offsets"], d["W1"], d["W3"], d["W2"])
    got = moe.ffn_train_backward(dY, ck, d["offsets"], d["W1"], d["W3"], d["W2"])
    torch.cuda.synchronize()
    sub = {w: d[w].cpu() for w in ("W1", "W3", "W2")} | {
        "X": d["X"][last].cpu(), "dY": dY[last].cpu(), "k": 1, "w": None, "row_src": None, "assign_row": None,
        "offsets": np.array([0, n])}
    part = moe.FFNCheckpoint(*(t[last] for t in ck))
    _check_forward(sub, Yp[last], part)
    _check_backward(sub, part, (got[0][last], got[1][last], *got[2:]))
    assert not got[0][:T - n].any() and not got[1][:T - n].any()


def test_ffn_train_column_tiles_of_many_experts():
    """1024 experts of 2^20 columns, the last four with a row each: the row and
    column tiles that the gate and up product could have, times their threads,
    do not fit 32 bits. (The three weight matrices share one buffer: only the
    last experts' are read.)"""
    T, H, F, E = 4, 32, 1 << 20, 1024
    say(f"[limits] ffn T={T} H={H} F={F} E={E}")
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of free memory")
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.empty(E * H * F, dtype=torch.bfloat16, device="cuda")
    last = 0.05 * torch.randn(T * H * F, generator=g, device="cuda", dtype=torch.bfloat16)
    W[-T * H * F:] = last
    X = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    offsets = torch.clamp(torch.arange(E + 1, dtype=torch.int32, device="cuda") - (E - T), min=0)
    Yp, ck = moe.ffn_train_forward(X, offsets, W.view(E, H, F), W.view(E, H, F), W.view(E, F, H))
    torch.cuda.synchronize()
    last = last.cpu()
    sub = {"X": X.cpu(), "W1": last.view(T, H, F), "W3": last.view(T, H, F), "W2": last.view(T, F, H), "k": 1,
           "row_src": None, "offsets": np.arange(T + 1)}
    _check_forward(sub, Yp, ck)
