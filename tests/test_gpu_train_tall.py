"""GPU: the expert FFN's training passes where they take 256-row tiles.

The tile height follows from the sizes of the whole pass (the rows of an expert
on average, and row tiles times the fewer column tiles of the pass's two
products), so each case first asks the library which kernels it takes, and for the split cases works out that their last round is
split. The oracle is the definition in 64 bits on the GPU; bounds are formed
from its own terms: u = 2^-24 for each fp32 operation of a sum (at most its
length times u times the sum of magnitudes), half = 2^-8 for each rounding to
bf16, 2^-4 (or half the smallest step, 2^-10 of the scale) for a checkpoint."""
import ctypes

import pytest
import torch

import mixture_experts_layer_count_amd as moe
from mixture_experts_layer_count_amd import _lib
from _gpu import say

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()
    yield
    torch.cuda.empty_cache()


def plan(T, H, F, E, k):
    """(forward rows, backward rows, persistent down product)"""
    v = [ctypes.c_int(-1) for _ in range(3)]
    assert moe.lib().moe_ffn_train_plan(T, k, E, H, F, *(ctypes.byref(x) for x in v)) == 0
    return v[0].value, v[1].value, bool(v[2].value)


def _case(T, H, F, E, k, skew, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    d = {"X": bf(T, H), "dY": bf(T, H), "W1": bf(E, H, F).mul_(0.05), "W3": bf(E, H, F).mul_(0.05),
         "W2": bf(E, F, H).mul_(0.05), "k": k, "w": None, "row_src": None, "assign_row": None}
    if E == 1:
        return d | {"offsets": torch.tensor([0, T], dtype=torch.int32, device="cuda")}
    z = torch.randn(T, E, generator=g, device="cuda") - skew * torch.arange(E, device="cuda")
    top, idx = torch.topk(z, k, dim=1)
    _, off, src, inv, _ = moe.permute(idx.int(), E)
    return d | {"w": torch.softmax(top, 1), "offsets": off, "row_src": src, "assign_row": inv}


def _forward(d):
    return moe.ffn_train_forward(d["X"], d["offsets"], d["W1"], d["W3"], d["W2"], row_src=d["row_src"], k=d["k"])


def _backward(d, ck, **kw):
    return moe.ffn_train_backward(d["dY"], ck, d["offsets"], d["W1"], d["W3"], d["W2"], topk_w=d["w"],
                                  row_src=d["row_src"], assign_row=d["assign_row"], **kw)


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out, worst {(err / tol.clamp(min=1e-300)).max():.3g} of the bound"


def _held(q, s):
    return q.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(32, 1)


def _experts(d):
    """(expert, its rows, their tokens, their assignments)"""
    off = d["offsets"].tolist()
    src = torch.arange(off[-1], device="cuda") if d["row_src"] is None else d["row_src"].long()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            yield e, slice(lo, hi), src[lo:hi] // d["k"], src[lo:hi]


def check_forward(d, Yp, ck):
    H, F = d["W1"].shape[1:]
    for e, r, t, _ in _experts(d):
        x = d["X"][t].double()
        v, err = {}, {}
        for n, w in (("g", "W1"), ("u", "W3")):
            m = d[w][e].double()
            v[n], err[n] = x @ m, H * U * (x.abs() @ m.abs())
            q, s = getattr(ck, n + "q")[r], getattr(ck, n + "s")[r]
            least = torch.exp2(s.double() - 127 - 10).repeat_interleave(32, 1)
            within(_held(q, s), v[n], torch.maximum(v[n].abs() * 2.0 ** -4, least) + err[n] * (1 + 2.0 ** -4),
                   f"checkpoint {n} of expert {e}")
        g, u = v["g"], v["u"]
        sg = 1 / (1 + torch.exp(-g))
        h = g * sg * u
        # |d silu| <= 1.1; silu by the hardware exp2 and reciprocal: 8 u (1 + |g|); then h to bf16
        dh = (g * sg).abs() * err["u"] + 1.1 * u.abs() * err["g"] + 8 * U * (1 + g.abs()) * h.abs()
        W2 = d["W2"][e].double()
        y, aw = h @ W2, W2.abs()
        within(Yp[r], y, HALF * y.abs() + (HALF + F * U) * (h.abs() @ aw) + 1.01 * (dh @ aw), f"Yp of expert {e}")


def check_backward(d, ck, got):
    """Gradients against the formulas on the checkpoint's own values."""
    k, (T, H), F = d["k"], d["dY"].shape, d["W1"].shape[2]
    dX, dw, dW1, dW3, dW2 = got
    xv = _held(ck.xq, ck.xs)
    rX, tX = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2))
    rw, tw = (torch.zeros(T * k, dtype=torch.float64, device="cuda") for _ in range(2))
    for e, r, t, a in _experts(d):
        g, u, dy, x = _held(ck.gq[r], ck.gs[r]), _held(ck.uq[r], ck.us[r]), d["dY"][t].double(), xv[t]
        w = 1.0 if d["w"] is None else d["w"].reshape(-1)[a].double().unsqueeze(1)
        W1, W3, W2 = (d[n][e].double() for n in ("W1", "W3", "W2"))
        p, dp = dy @ W2.T, H * U * (dy.abs() @ W2.abs().T)
        sg = 1 / (1 + torch.exp(-g))
        h, hu, hg = g * sg * u, g * sg, u * (sg + g * sg * (1 - sg))
        # the sigmoid and the few products that follow; |hg| by magnitudes, its bracket may cancel
        rnd = 16 * U * (1 + g.abs())
        mg = u.abs() * sg * (1 + g.abs() * (1 - sg))
        ap, ah = p.abs(), h.abs()
        rw[a] = (p * h).sum(1)
        tw[a] = (dp * ah + (rnd + F * U) * ap * ah).sum(1)
        dg, du = w * p * hg, w * p * hu
        eg = HALF * dg.abs() + 1.01 * w * (hg.abs() * dp + rnd * ap * mg)
        eu = HALF * du.abs() + 1.01 * w * (hu.abs() * dp + rnd * ap * hu.abs())
        rX.index_add_(0, t, dg @ W1.T + du @ W3.T)
        n = (2 * F + k) * U
        tX.index_add_(0, t, (eg + n * dg.abs()) @ W1.abs().T + (eu + n * du.abs()) @ W3.abs().T)
        m = (g.shape[0]) * U * 1.01
        ax = x.abs().T
        for name, out, ref, tol in (("dW1", dW1, x.T @ dg, ax @ (eg + m * dg.abs())),
                                    ("dW3", dW3, x.T @ du, ax @ (eu + m * du.abs())),
                                    ("dW2", dW2, (w * h).T @ dy, ((HALF + m + 1.01 * rnd) * w * ah).T @ dy.abs())):
            within(out[e], ref, HALF * ref.abs() + 1.01 * tol + 1e-30, f"{name} of expert {e}")
    within(dX, rX, HALF * rX.abs() + 1.01 * tX, "dX")
    within(dw.reshape(-1), rw, tw + 1e-30, "dtopk_w")


def _split(d, cols, steps):
    """Parts of an item of the last round of a product with `cols` column tiles
    and so many steps, on 256-row tiles."""
    off = d["offsets"].tolist()
    tiles = sum((hi - lo + 255) // 256 for lo, hi in zip(off, off[1:]))
    tail = (tiles * cols + 7) // 8 % 32  # items of an XCD beyond whole rounds of its 32 CUs
    return max(1, min(4, 32 // tail, steps // 32)) if tail else 1


CASES = [
    # T, H, F, E, k, skew, (forward rows, backward rows, persistent down), parts of a split item by product
    # half steps (H and F % 64 = 32), three and more column tiles, the last ones part full, experts of a few to many rows
    (17000, 544, 608, 7, 2, 0.8, (256, 256, False), {}),
    (40000, 288, 352, 1, 1, 0.0, (256, 256, False), {}),      # in row order
    # the persistent down product
    (16500, 512, 320, 4, 2, 0.3, (256, 256, True), {}),
    (4200, 2048, 1024, 4, 2, 0.1, (256, 256, True), {}),
    # 256 rows in one pass only: by the tiles (forward 192, backward 96), by the rows (256 an expert)
    (6000, 1024, 512, 4, 2, 0.1, (256, 128, True), {}),
    (16384, 512, 512, 64, 1, 0.0, (256, 128, True), {}),
    # sums long enough for a split last round: over H, and over F
    (22000, 4128, 800, 4, 1, 0.1, (256, 256, False), {"GATE_UP": 2, "BACK": 2}),
    (33000, 288, 4128, 3, 1, 0.1, (256, 256, False), {"DOWN": 2, "DX": 4}),
]


@pytest.mark.parametrize("T,H,F,E,k,skew,kernels,parts", CASES)
def test_ffn_train_tall_tiles(T, H, F, E, k, skew, kernels, parts):
    say(f"[train tall] ffn T={T} H={H} F={F} E={E} k={k} skew={skew}")
    assert plan(T, H, F, E, k) == kernels
    d = _case(T, H, F, E, k, skew)
    tiles = lambda n, w: (n + w - 1) // w  # noqa: E731
    product = {"GATE_UP": (tiles(F, 128), tiles(H, 64)), "DOWN": (tiles(H, 256), tiles(F, 64)),
               "BACK": (tiles(F, 256), tiles(H, 64)), "DX": (tiles(H, 256), 2 * tiles(F, 64))}
    assert {n: _split(d, *product[n]) for n in parts} == parts
    Yp, ck = _forward(d)
    check_forward(d, Yp, ck)
    got = _backward(d, ck)
    check_backward(d, ck, got)
    # identical run to run
    Yp2, ck2 = _forward(d)
    assert torch.equal(Yp, Yp2) and all(torch.equal(a, b) for a, b in zip(ck, ck2))
    assert all(torch.equal(a, b) for a, b in zip(got, _backward(d, ck)))
