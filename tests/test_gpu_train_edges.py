"""GPU: values and calls at the edges of what the training operators document."""
import pytest
import torch

import mixture_experts_layer_count_amd as moe
from _gpu import say
from test_gpu_train import _check_router, _router

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


@pytest.mark.parametrize("F", [32, 96, 160, 288, 480])
def test_infinite_gradient_beside_part_full_columns(F):
    """A column tile that the matrix ends inside holds columns that do not
    exist. An infinite dY with positive weights and activations makes the
    routing weight's gradient +inf, and every other output what the formula
    says; the missing columns add nothing (not inf * 0)."""
    say(f"[train edges] infinite dY, F={F}")
    T, H = 20, 64
    g = torch.Generator().manual_seed(F)
    pos = lambda *s: (0.1 + torch.rand(*s, generator=g)).bfloat16().cuda()  # noqa: E731
    X, W1, W3, W2, dY = pos(T, H), pos(1, H, F), pos(1, H, F), pos(1, F, H), pos(T, H)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    _, ck = moe.ffn_train_forward(X, off, W1, W3, W2)
    t = 7
    dY[t, 3] = float("inf")
    dX, dw, dW1, dW3, dW2 = moe.ffn_train_backward(dY, ck, off, W1, W3, W2)
    rest = [i for i in range(T) if i != t]
    # g, u > 0: p, dg and du are +inf in every column, and so are their sums
    assert torch.isfinite(dw[rest]).all() and torch.isfinite(dX[rest]).all()
    assert (dw[t] == float("inf")).all() and (dX[t] == float("inf")).all()
    assert (dW1 == float("inf")).all() and (dW3 == float("inf")).all()
    assert (dW2[0, :, 3] == float("inf")).all()
    assert torch.isfinite(dW2[0][:, [i for i in range(H) if i != 3]]).all()


def test_weight_gradient_buffers_come_in_threes():
    """dW is (dW1, dW3, dW2): another number of buffers is refused by name, and
    nothing is added to any of them."""
    say("[train edges] dW of two and of four buffers")
    T, H, F = 8, 64, 32
    g = torch.Generator().manual_seed(1)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    X, W1, W3, W2, dY = bf(T, H), bf(1, H, F), bf(1, H, F), bf(1, F, H), bf(T, H)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    _, ck = moe.ffn_train_forward(X, off, W1, W3, W2)
    bufs = [torch.ones_like(w) for w in (W1, W3, W2, W1)]
    for n in (0, 1, 2, 4):
        with pytest.raises(ValueError, match="dW1, dW3, dW2"):
            moe.ffn_train_backward(dY, ck, off, W1, W3, W2, dW=bufs[:n])
    torch.cuda.synchronize()
    assert all((b == 1).all() for b in bufs)


def test_scale_byte_of_no_number():
    """E8M0's byte 255 stands for no number: every value under it is NaN."""
    say("[train edges] scale byte 255")
    Q = torch.arange(256, dtype=torch.uint8).reshape(8, 32).cuda()
    S = torch.full((8, 1), 255, dtype=torch.uint8, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        assert torch.isnan(moe.checkpoint_unpack(Q, S, dt)).all()


@pytest.mark.parametrize("seq", [
    [0] * 40 + [7] * 30 + [8] * 3 + [60] * 50 + [97] * 200,     # empty ones first, between and last; 3 tokens behind
    [5] * 20 + [5, 40] + [40] * 300,                            # tokens in front of all, 60 behind
    [0, 100] + [100] * 500, [50] * 400, [0] * 100 + [100] * 100,
])
def test_router_losses_many_empty_sequences(seq):
    say(f"[train edges] router losses, {len(seq) - 1} sequences, few of them with tokens")
    _check_router(*_router(100, 16, 3, len(seq)), seq)


def test_router_losses_padded_batch_time():
    """A batch padded to a fixed number of sequences, with padding tokens behind
    them, takes about as long as one whose last sequence reaches the end: the
    empty sequences are not walked one by one (that took 6 and 35 times as
    long)."""
    say("[train edges] router losses of a padded batch, time")
    T, E, k, B = 8192, 128, 8, 4096
    z, idx, w, dw = (t.cuda() for t in _router(T, E, k, 3))

    def times(last):
        seq = torch.tensor([last * i // 8 for i in range(9)] + [last] * (B - 8), dtype=torch.int32, device="cuda")
        per = moe.balance_loss(z, idx, 0.1, 0.1, seq_offsets=seq)[2]
        out = []
        for f in (lambda: moe.balance_loss(z, idx, 0.1, 0.1, seq_offsets=seq),
                  lambda: moe.route_backward(z, idx, w, dw, per, 0.1, 0.1, seq_offsets=seq)):
            t = []
            for _ in range(7):
                a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                f()
                a.record()
                for _ in range(5):
                    f()
                b.record()
                torch.cuda.synchronize()
                t.append(a.elapsed_time(b))
            out.append(sorted(t)[3])
        return out

    times(T)
    for padded, whole in zip(times(T - 191), times(T)):
        assert padded < 3 * whole
