"""GPU: the training operators against the fp64 oracle (oracle/train.py).

Tolerances are error bounds, formed per element from the oracle's own terms
before any run: u = 2^-24 for each fp32 operation of a sum (at most its length
times u times the sum of magnitudes), half = 2^-8 for each rounding to bf16 (an
operand of a matrix product, or an output), and
e4m3 = 2^-4 (or half the smallest step, 2^-10 of the scale) for a checkpoint."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_count_amd as moe
import oracle
from mixture_experts_layer_count_amd import _lib
from oracle import train
from _gpu import say

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out, worst {np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} of the bound"


# ----------------------------------------------------------------------------
# checkpoints
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("R,C,ld,dt", [(1, 32, 32, torch.bfloat16), (3, 96, 104, torch.bfloat16),
                                       (257, 544, 544, torch.bfloat16), (130, 2048, 2048, torch.bfloat16),
                                       (5, 64, 68, torch.float32), (33, 1408, 1408, torch.float32)])
def test_checkpoint_bit_exact(R, C, ld, dt):
    say(f"[train] checkpoint {R} x {C} (rows of {ld}) {dt}")
    g = torch.Generator().manual_seed(R + C)
    x = torch.randn(R, ld, generator=g) * torch.exp2(torch.randint(-30, 30, (R, 1), generator=g).float())
    x[0, :32] = 0.0
    x = x.to(dt)
    if R > 2:
        x[1, :32] = torch.tensor(448.0).to(dt)                       # fits its scale exactly
        x[1, 0] = 1e-30                                              # rounds to zero
        x[2, :8] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1, -1, 3e38, -1e-38, 0]).to(dt)
    X = x.cuda()[:, :C]
    Q, S = moe.checkpoint_pack(X)
    q, s = train.checkpoint_pack(f64(X))
    np.testing.assert_array_equal(S.cpu().numpy(), s)
    got, nan = Q.cpu().numpy(), np.isnan(train.checkpoint_values(q, s))
    np.testing.assert_array_equal(got[~nan], q[~nan])
    np.testing.assert_array_equal(got[nan] & 0x7f, 0x7f)
    for out in (torch.bfloat16, torch.float32):
        np.testing.assert_array_equal(f64(moe.checkpoint_unpack(Q, S, out)), train.checkpoint_values(q, s))


def test_checkpoint_strided_and_empty():
    say("[train] checkpoint of a view with gaps between rows, of one row, of none")
    x = torch.randn(9, 3 * 160, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    view = x.view(9, 3, 160)[:, 1, :96]
    Q, S = moe.checkpoint_pack(view)
    q, s = moe.checkpoint_pack(view.contiguous())
    assert torch.equal(Q, q) and torch.equal(S, s)
    Q, S = moe.checkpoint_pack(view[4:5])
    assert torch.equal(Q, q[4:5]) and torch.equal(S, s[4:5])
    Q, S = moe.checkpoint_pack(x[:0])
    assert Q.shape == (0, 480) and S.shape == (0, 15) and moe.checkpoint_unpack(Q, S).shape == (0, 480)
    with pytest.raises(moe.MoEError):
        moe.checkpoint_pack(x[:1].expand(9, 480))       # rows on top of each other
    with pytest.raises(moe.MoEError):
        moe.checkpoint_pack(x.view(-1)[4:4 + 480].view(5, 96))  # off the 16-byte boundary


def test_checkpoint_every_code():
    Q = torch.arange(256, dtype=torch.uint8).reshape(8, 32).cuda()
    S = torch.tensor([[120], [127], [1], [10], [200], [240], [127], [64]], dtype=torch.uint8).cuda()
    ref = train.checkpoint_values(Q.cpu().numpy(), S.cpu().numpy())
    ref[np.abs(ref) < 2.0 ** -126] = 0.0                             # below the smallest normal: may be flushed
    for out in (torch.bfloat16, torch.float32):
        got = f64(moe.checkpoint_unpack(Q, S, out))
        got[np.abs(got) < 2.0 ** -126] = 0.0
        np.testing.assert_array_equal(got, ref)


# ----------------------------------------------------------------------------
# router losses
# ----------------------------------------------------------------------------
def _router(T, E, k, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    z = scale * torch.randn(T, E, generator=g)
    w, idx = torch.topk(z, k, dim=1)
    return z, idx.int(), torch.softmax(w, 1), torch.randn(T, k, generator=g)


def _check_router(z, idx, w, dw, seq, alpha=0.3, beta=0.2, dloss=(0.7, -1.5)):
    T, E = z.shape
    seq_d = None if seq is None else torch.tensor(seq, dtype=torch.int32).cuda()
    zd, id_, wd, dwd = z.cuda(), idx.cuda(), w.cuda(), dw.cuda()
    loss, counts, per = moe.balance_loss(zd, id_, alpha, beta, seq_offsets=seq_d)
    d = moe.route_backward(zd, id_, wd, dwd, per, alpha, beta, seq_offsets=seq_d,
                           dloss=torch.tensor(dloss).cuda())
    zn, ix = f64(z), idx.numpy()
    ref_loss, ref_counts, ref_per = train.balance_loss(zn, ix, alpha, beta, seq)
    np.testing.assert_array_equal(counts.cpu().numpy(), ref_counts)
    np.testing.assert_array_equal(per.cpu().numpy(), ref_per)
    # p: 4 u from exp, the sum over E and the division, E u in all at most; the
    # sum over tokens: at most 64 in a lane, 6 + 4 steps in a block, T / 16 / 16
    # chunks in a wavefront, 16 wavefronts; positive terms, so relative
    rel = (E + 64 + 32 + T / 256 + 16) * U
    lse2 = (train.log_sum_exp(zn) ** 2)
    # lse = top + log(sum): u of each, absolute where they cancel
    top = np.abs(np.where(np.isneginf(zn.max(1)), 0, zn.max(1)))
    lse_err = (E + 8) * U + 4 * U * (top + np.sqrt(lse2))
    z_err = beta * (2 * np.sqrt(lse2) * lse_err + 4 * U * lse2).mean() + rel * abs(ref_loss[1])
    within(loss, ref_loss, np.array([rel * abs(ref_loss[0]), z_err]) + 1e-30, "loss")
    # each of the three terms by the magnitudes it adds
    a = train.route_backward(zn, ix, alpha=alpha, beta=0.0, seq=seq, dloss=dloss)
    f = E * ref_per.max(initial=0) / 1.0
    p = train.probabilities(zn)
    seqs = [0, T] if seq is None else seq
    mag = np.zeros_like(zn)
    live = sum(hi > lo for lo, hi in zip(seqs, seqs[1:]))
    n_all = sum(hi - lo for lo, hi in zip(seqs, seqs[1:]))
    for b, (lo, hi) in enumerate(zip(seqs, seqs[1:])):
        if hi > lo:
            fb = E * ref_per[b] / (idx.shape[1] * (hi - lo))
            q = p[lo:hi]
            mag[lo:hi] += abs(dloss[0]) * alpha / (live * (hi - lo)) * q * (fb + (q * fb).sum(1, keepdims=True))
            le = np.sqrt(lse2[lo:hi])[:, None]
            mag[lo:hi] += abs(dloss[1]) * 2 * beta / n_all * q * (le + (lse_err[lo:hi] / ((E + 16) * U))[:, None])
    wn, dwn = f64(w), f64(dw)
    vm = wn * (np.abs(dwn) + (wn * np.abs(dwn)).sum(1, keepdims=True))
    for t in range(T):
        for j in range(idx.shape[1]):
            if 0 <= ix[t, j] < E:
                mag[t, ix[t, j]] += vm[t, j]
    ref = train.route_backward(zn, ix, wn, dwn, alpha, beta, seq, dloss)
    within(d, ref, (E + 16 + 2 * idx.shape[1]) * U * mag + 1e-30, "dlogits")
    return loss, counts, per, d


@pytest.mark.parametrize("T,E,k,seq", [
    (1, 1, 1, None), (1, 8, 2, None), (5, 4, 4, None), (64, 8, 2, [0, 64]), (70, 8, 8, [0, 1, 1, 33, 70]),
    (33, 7, 3, [0, 10, 33]), (50, 16, 2, [5, 20, 41]), (130, 12, 5, None), (100, 32, 8, [0, 0, 100]),
    (257, 60, 6, [0, 100, 200, 257]), (300, 64, 8, None), (90, 65, 4, [0, 45, 90]), (513, 128, 8, [0, 17, 511, 513]),
    (90, 130, 9, None), (200, 256, 8, [0, 64, 128, 200]), (40, 320, 20, None), (33, 1024, 64, None),
    (20, 333, 64, [0, 7, 20]), (3000, 40, 4, [0, 1500, 3000]),
])
def test_router_losses(T, E, k, seq):
    say(f"[train] router losses T={T} E={E} k={k} seq={seq}")
    _check_router(*_router(T, E, k, T + E), seq)


def test_router_losses_masks():
    say("[train] router losses: masked experts, masked rows, lowest values, stray picks")
    z, idx, w, dw = _router(200, 24, 3, 5)
    z[:, 3] = -float("inf")                      # an expert nobody may pick
    z[::7, 8:] = -float("inf")
    z[11] = -float("inf")                        # a row that nothing is left of
    z[12, :20] = torch.finfo(torch.float32).min  # the type's lowest value as the mask
    z[13] = 80.0                                 # far from zero
    w, idx = torch.topk(z, 3, dim=1)
    w, idx = torch.softmax(w, 1), idx.int()
    w[11] = 1 / 3
    idx[20, 1] = -1                              # picks of a padded token
    idx[21] = 24
    idx[22] = idx[22, 0]                         # the same expert three times
    _, _, _, d = _check_router(z, idx, w, dw, [0, 60, 60, 150])
    assert torch.isfinite(d).all()
    # a NaN stays in its row of the gradient, and shows in the losses
    z[30, 4] = float("nan")
    zd = z.cuda()
    loss, _, per = moe.balance_loss(zd, idx.cuda(), 0.1, 0.1)
    assert torch.isnan(loss).all()
    d = moe.route_backward(zd, idx.cuda(), seq_counts=per, alpha=0.1, beta=0.1)
    assert torch.isnan(d[30]).all() and torch.isfinite(torch.cat([d[:30], d[31:]])).all()


def test_router_terms_apart():
    say("[train] route_backward: each term alone; no tokens")
    z, idx, w, dw = _router(100, 20, 4, 9)
    zd, ix, wd, dwd = z.cuda(), idx.cuda(), w.cuda(), dw.cuda()
    _, _, per = moe.balance_loss(zd, ix, 0.3, 0.2)
    aux = moe.route_backward(zd, ix, seq_counts=per, alpha=0.3, beta=0.2)
    only = moe.route_backward(zd, ix, wd, dwd)
    both = moe.route_backward(zd, ix, wd, dwd, per, 0.3, 0.2)
    # the two terms are added last: one rounding
    within(both, f64(aux) + f64(only), 2 * U * (np.abs(f64(aux)) + np.abs(f64(only))) + 1e-30, "sum of terms")
    within(only, train.route_backward(f64(z), idx.numpy(), f64(w), f64(dw), aux=False),
           16 * U * (np.abs(f64(dw)).max() + 1) * 2, "routing term")
    loss, counts, per = moe.balance_loss(zd[:0], ix[:0], 0.3, 0.2)
    assert loss.tolist() == [0.0, 0.0] and not counts.any() and not per.any()
    assert moe.route_backward(zd[:0], ix[:0], wd[:0], dwd[:0]).shape == (0, 20)
    # logits off the 16-byte boundary take the scalar loads
    off = torch.empty(100 * 20 + 1, device="cuda")[1:].view(100, 20)
    off.copy_(zd)
    l0, l1 = moe.balance_loss(zd, ix, 0.3, 0.2)[0], moe.balance_loss(off, ix, 0.3, 0.2)[0]
    within(l1, f64(l0), 300 * U * np.abs(f64(l0)), "unaligned logits")


# ----------------------------------------------------------------------------
# expert FFN
# ----------------------------------------------------------------------------
def _ffn_case(T, H, F, E, k, seed=0, gathered=True, skew=0.0):
    g = torch.Generator().manual_seed(seed + T + H)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    c = {"X": bf(T, H), "dY": bf(T, H), "W1": (0.05 * bf(E, H, F).float()).bfloat16(),
         "W3": (0.05 * bf(E, H, F).float()).bfloat16(), "W2": (0.05 * bf(E, F, H).float()).bfloat16(), "k": k}
    if gathered:
        z = torch.randn(T, E, generator=g) - skew * torch.arange(E)
        w, idx = torch.topk(z, k, dim=1)
        c["w"] = torch.softmax(w, 1)
        _, off, src, inv = oracle.permute(idx.numpy(), E)
        c |= {"offsets": off, "row_src": src, "assign_row": inv}
    else:
        cut = np.sort(np.random.default_rng(seed).integers(0, T + 1, size=E - 1))
        c |= {"offsets": np.concatenate([[0], cut, [T]]), "row_src": None, "assign_row": None, "w": None}
    return c


def _dev(c):
    i32 = lambda a: None if a is None else torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()  # noqa: E731
    return {n: (v.cuda() if isinstance(v, torch.Tensor) else v if n == "k" else i32(v)) for n, v in c.items()}


def _forward(d, **kw):
    return moe.ffn_train_forward(d["X"], d["offsets"], d["W1"], d["W3"], d["W2"], row_src=d["row_src"], k=d["k"], **kw)


def _backward(d, ck, **kw):
    return moe.ffn_train_backward(d["dY"], ck, d["offsets"], d["W1"], d["W3"], d["W2"], topk_w=d["w"],
                                  row_src=d["row_src"], assign_row=d["assign_row"], **kw)


def _check_forward(c, Yp, ck):
    X, W1, W3, W2 = (f64(c[n]) for n in ("X", "W1", "W3", "W2"))
    H, F = W1.shape[1:]
    k, off = c["k"], c["offsets"]
    M = int(off[-1])
    src = np.arange(M) if c["row_src"] is None else c["row_src"]
    q, s = train.checkpoint_pack(X)
    np.testing.assert_array_equal(ck.xq.cpu().numpy(), q)
    np.testing.assert_array_equal(ck.xs.cpu().numpy(), s)
    held = {n: train.checkpoint_values(getattr(ck, n + "q").cpu().numpy(), getattr(ck, n + "s").cpu().numpy()) for n in "gu"}
    exps = {n: getattr(ck, n + "s").cpu().numpy().astype(np.float64) - 127 for n in "gu"}
    for e in range(len(off) - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        x = X[src[lo:hi] // k]
        v = {"g": x @ W1[e], "u": x @ W3[e]}
        err = {"g": H * U * (np.abs(x) @ np.abs(W1[e])), "u": H * U * (np.abs(x) @ np.abs(W3[e]))}
        for n in "gu":
            sc = exps[n][lo:hi]
            step = np.maximum(np.abs(v[n]) * 2.0 ** -4, np.repeat(np.exp2(sc - 10), 32, axis=1))
            within(held[n][lo:hi], v[n], step + err[n] * (1 + 2.0 ** -4), f"checkpoint {n} of expert {e}")
            top = np.abs(v[n]).reshape(hi - lo, -1, 32).max(axis=2)
            slack = err[n].reshape(hi - lo, -1, 32).max(axis=2)
            assert (top - slack <= 448 * np.exp2(sc)).all() and (top + slack > 224 * np.exp2(sc)).all()
        h, hu, hg = train.swiglu_backward(v["g"], v["u"])
        # silu by the hardware exp2 and reciprocal: 8 u (1 + |g|); then h to bf16
        dh = np.abs(hu) * err["u"] + 1.1 * np.abs(v["u"]) * err["g"] + 8 * U * (1 + np.abs(v["g"])) * np.abs(h)
        y = h @ W2[e]
        mag = np.abs(h) @ np.abs(W2[e])
        within(f64(Yp)[lo:hi], y, HALF * np.abs(y) + (HALF + F * U) * mag + 1.01 * (dh @ np.abs(W2[e])), f"Yp of expert {e}")


def _check_backward(c, ck, got, base=None, half_out=HALF):
    """Gradients against the oracle on the checkpoint's own values."""
    dY, W1, W3, W2 = (f64(c[n]) for n in ("dY", "W1", "W3", "W2"))
    k, off = c["k"], c["offsets"]
    T, H = dY.shape
    M, F = int(off[-1]), W1.shape[2]
    val = lambda n: train.checkpoint_values(getattr(ck, n + "q").cpu().numpy(), getattr(ck, n + "s").cpu().numpy())  # noqa: E731
    x, g, u = val("x"), val("g")[:M], val("u")[:M]
    r = train.ffn_backward(dY, x, g, u, None if c["w"] is None else f64(c["w"]), c["row_src"], off, W1, W3, W2, k)
    w, src = r["w"][:, None], r["src"]
    tol = {"dX": np.zeros((T, H)), "dw": np.zeros(T * k), "dW1": np.zeros_like(r["dW1"]),
           "dW3": np.zeros_like(r["dW3"]), "dW2": np.zeros_like(r["dW2"])}
    rnd = U * 16 * (1 + np.abs(g))                     # sigmoid and the few products that follow it
    for e in range(len(off) - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        t, s = src[lo:hi] // k, slice(lo, hi)
        dp = H * U * (np.abs(dY[t]) @ np.abs(W2[e]).T)
        p, h = np.abs(r["p"][s]), np.abs(r["h"][s])
        tol["dw"][src[s]] = (dp * h + (rnd[s] + F * U) * p * h).sum(1)
        # |du s (1 + g (1 - s))| by magnitudes: the bracket may cancel
        sg = 1 / (1 + np.exp(-g[s]))
        mg = np.abs(u[s]) * sg * (1 + np.abs(g[s]) * (1 - sg))
        row = {}
        for n, cf, mag in (("dW1", np.abs(r["hg"][s]), mg), ("dW3", np.abs(r["hu"][s]), np.abs(r["hu"][s]))):
            full = w[s] * p * cf
            row[n] = (HALF * full + 1.01 * w[s] * (cf * dp + rnd[s] * p * mag), full)
        for n, wt in (("dW1", W1[e]), ("dW3", W3[e])):
            d, full = row[n]
            np.add.at(tol["dX"], t, d @ np.abs(wt).T + (2 * F + k) * U * (full @ np.abs(wt).T))
            xt = np.abs(x[t]).T
            tol[n][e] = xt @ d + (hi - lo) * U * 1.01 * (xt @ full)
        wh = w[s] * h
        tol["dW2"][e] = ((HALF + (hi - lo) * U) * wh + 1.01 * rnd[s] * wh).T @ np.abs(dY[t])
    dX, dw, dW1, dW3, dW2 = got
    add = 0.0 if base is None or "dX" not in base else base["dX"]
    if dX is not None:
        ref = r["dX"] + add
        within(dX, ref, HALF * np.abs(ref) + 1.01 * tol["dX"] + 4 * U * np.abs(add), "dX")
    if dw is not None:
        within(dw, r["dw"], tol["dw"].reshape(T, k) + 1e-30, "dtopk_w")
    for n, v in (("dW1", dW1), ("dW3", dW3), ("dW2", dW2)):
        if v is None:
            continue
        ref = r[n] + (0.0 if base is None or n not in base else base[n])
        within(v, ref, half_out * np.abs(ref) + 1.01 * tol[n] + 1e-30, n)


FFN_CASES = [
    # T, H, F, E, k, gathered, skew
    (1, 32, 32, 1, 1, False, 0), (1, 64, 32, 4, 2, True, 0), (2, 96, 160, 3, 3, True, 0), (37, 96, 160, 12, 2, True, 0),
    (64, 544, 96, 4, 2, True, 0), (130, 256, 256, 2, 1, False, 0), (300, 160, 416, 8, 3, True, 0.5),
    (700, 320, 288, 4, 2, True, 1.5), (513, 288, 64, 2, 2, True, 0), (129, 64, 544, 64, 8, True, 0),
    (1000, 96, 96, 3, 1, True, 30.0),   # every token to one expert, the others empty
    (4700, 64, 32, 1, 1, False, 0),     # more rows than one window of row numbers
    (4300, 32, 64, 2, 2, True, 0),
    # 256-row tiles: gate/up and dH; dX; a short down projection
    # (128-row tiles by now: the height follows from both products of a pass; test_gpu_train_tall.py has 256)
    (8200, 128, 2080, 2, 1, True, 0.3), (8200, 2080, 128, 2, 1, True, 0.3), (8200, 2048, 160, 2, 1, False, 0),
    # sums long enough for a split tail: gate/up and dH over H (2 and 4 parts), down and dX over F
    (200, 4128, 64, 2, 1, True, 0), (70, 8256, 96, 2, 2, True, 0), (150, 64, 4160, 2, 2, True, 0.5),
    # the most experts, the most picks
    (60, 64, 96, 1024, 4, True, 0), (9, 32, 64, 70, 64, True, 0),
    # several weight-gradient tiles for each workgroup, experts of 0 to 4 steps
    (190, 1056, 1120, 12, 2, True, 0.4),
]


@pytest.mark.parametrize("T,H,F,E,k,gathered,skew", FFN_CASES)
def test_ffn_train(T, H, F, E, k, gathered, skew):
    say(f"[train] ffn T={T} H={H} F={F} E={E} k={k} gathered={gathered} skew={skew}")
    c = _ffn_case(T, H, F, E, k, gathered=gathered, skew=skew)
    d = _dev(c)
    Yp, ck = _forward(d)
    torch.cuda.synchronize()
    _check_forward(c, Yp, ck)
    got = _backward(d, ck)
    _check_backward(c, ck, got)
    # identical run to run
    again = _backward(d, ck)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # a part of the outputs alone is the same part
    dX, dw, dW1, dW3, dW2 = _backward(d, ck, need=("dX",))
    assert torch.equal(dX, got[0]) and dw is None and dW1 is None
    dX, dw, dW1, dW3, dW2 = _backward(d, ck, need=("dtopk_w", "dW"))
    assert dX is None and torch.equal(dw, got[1]) and torch.equal(dW1, got[2]) and torch.equal(dW2, got[4])


@pytest.mark.parametrize("T,H,F,E,skew", [(200, 160, 96, 6, 0.7), (120, 1056, 800, 11, 0.7)])
def test_ffn_train_accumulate(T, H, F, E, skew):
    say(f"[train] ffn gradients added to f32 and bf16 buffers, and to another path's dX: H={H} F={F} E={E}")
    c = _ffn_case(T, H, F, E, 2, skew=skew)
    d = _dev(c)
    _, ck = _forward(d)
    empty = np.diff(c["offsets"]) == 0
    for dt, half in ((torch.float32, 4 * U), (torch.bfloat16, HALF)):
        g = torch.Generator().manual_seed(4)
        base = {n: torch.randn(d[w].shape, generator=g).to(dt) for n, w in (("dW1", "W1"), ("dW3", "W3"), ("dW2", "W2"))}
        add = torch.randn(T, H, generator=g).bfloat16()
        bufs = tuple(base[n].cuda() for n in ("dW1", "dW3", "dW2"))
        out = add.cuda()
        got = _backward(d, ck, dW=bufs, dX_add=out)
        assert got[2] is bufs[0] and torch.equal(out.cpu(), add)
        _check_backward(c, ck, got, base={n: f64(v) for n, v in base.items()} | {"dX": f64(add)}, half_out=half)
        new = _backward(d, ck, dw_dtype=dt)
        _check_backward(c, ck, new, half_out=half)
        for e in np.nonzero(empty)[0]:
            assert torch.equal(bufs[0][e].cpu(), base["dW1"][e]) and not new[2][e].any() and not new[4][e].any()


def test_ffn_train_no_tokens():
    say("[train] ffn without tokens")
    c = _ffn_case(8, 64, 32, 3, 2)
    d = _dev(c)
    d |= {"X": d["X"][:0], "dY": d["dY"][:0], "w": d["w"][:0], "row_src": d["row_src"][:0],
          "assign_row": d["assign_row"][:0], "offsets": torch.zeros(4, dtype=torch.int32, device="cuda")}
    Yp, ck = _forward(d)
    assert Yp.shape == (0, 64)
    dX, dw, dW1, dW3, dW2 = _backward(d, ck)
    assert dX.shape == (0, 64) and dw.shape == (0, 2)
    assert not dW1.any() and not dW3.any() and not dW2.any()
    keep = tuple(torch.full_like(w, 2.0) for w in (d["W1"], d["W3"], d["W2"]))
    _backward(d, ck, dW=keep)
    assert all((v == 2.0).all() for v in keep)


def test_ffn_train_rows_behind_the_last_group():
    say("[train] rows behind the last group, and picks that were left out")
    T, H, F, E, k = 60, 96, 64, 5, 2
    c = _ffn_case(T, H, F, E, k)
    # the last group loses its rows: their picks were left out by the permutation
    full = c["offsets"].copy()
    c["offsets"] = full.copy()
    c["offsets"][E] = full[E - 1]
    m = int(c["offsets"][E])
    d = _dev(c)
    lib, M = moe.lib(), T * k
    ptr = lambda t: t.data_ptr()  # noqa: E731
    Yp = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
    bufs = [torch.full(s, 91, dtype=torch.uint8, device="cuda") for s in
            ((T, H), (T, H // 32), (M, F), (M, F // 32), (M, F), (M, F // 32))]
    ptrs = _lib._CheckpointPtrs(*(ptr(b) for b in bufs))
    ws = torch.empty(lib.moe_ffn_train_forward_workspace_bytes(T, k, E, H, F), dtype=torch.uint8, device="cuda")
    st = lib.moe_ffn_train_forward(ptr(d["X"]), ptr(d["row_src"]), k, T, ptr(d["offsets"]), E, H, F, ptr(d["W1"]),
                                   ptr(d["W3"]), ptr(d["W2"]), 1, ptr(Yp), _lib.ctypes.byref(ptrs), ptr(ws),
                                   ws.numel(), _lib._stream())
    assert st == 0
    ck = moe.FFNCheckpoint(*bufs)
    assert (Yp[m:] == 7.0).all() and all((b[m:] == 91).all() for b in bufs[2:])
    got = _backward(d, ck)
    # the oracle on the rows that are left
    c2 = dict(c)
    c2["row_src"] = c["row_src"][:m]
    _check_backward(c2, ck, got)
    dropped = c["row_src"][m:]
    assert not got[1].reshape(-1)[torch.as_tensor(dropped, device="cuda").long()].any()


def test_ffn_train_every_pick_left_out():
    say("[train] ffn whose permutation left every pick out")
    c = _ffn_case(40, 64, 96, 3, 2)
    d = _dev(c)
    _, ck = _forward(d)
    d["offsets"] = torch.zeros(4, dtype=torch.int32, device="cuda")
    Yp, _ = _forward(d)
    assert Yp.shape == (80, 64)
    dX, dw, dW1, dW3, dW2 = _backward(d, ck)
    assert not any(t.any() for t in (dX, dw, dW1, dW3, dW2))
    add = torch.randn(40, 64).bfloat16().cuda()
    assert torch.equal(_backward(d, ck, need=("dX",), dX_add=add)[0], add)


def _sub(c, ck, e, rows, tokens, cols=slice(None)):
    """Rows of expert e (and columns of F) as a problem of their own, k = 1 and
    in row order: its case and its checkpoint."""
    n = len(rows)
    groups = slice(None) if cols == slice(None) else slice(cols.start // 32, cols.stop // 32)
    sub = {"X": c["X"][tokens].cpu(), "dY": c["dY"][tokens].cpu(), "W1": c["W1"][e:e + 1, :, cols].cpu(),
           "W3": c["W3"][e:e + 1, :, cols].cpu(), "W2": c["W2"][e:e + 1, cols].cpu(), "k": 1,
           "w": c["w"].reshape(-1)[c["row_src"].long()[rows]].reshape(n, 1).cpu(), "offsets": np.array([0, n]),
           "row_src": None, "assign_row": None}
    part = moe.FFNCheckpoint(*(t[tokens] for t in ck[:2]), ck.gq[rows][:, cols], ck.gs[rows][:, groups],
                             ck.uq[rows][:, cols], ck.us[rows][:, groups])
    return sub, part


@pytest.mark.parametrize("T,H,F,E,k", [(70000, 64, 4096, 8, 8),     # 2.3e9 values of g
                                       (300, 8192, 4128, 64, 1)])   # 2.2e9 of a weight matrix
def test_ffn_train_past_32_bits(T, H, F, E, k):
    say(f"[train] ffn with offsets past 32 bits: T={T} H={H} F={F} E={E} k={k}")
    g = torch.Generator(device="cuda").manual_seed(T)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    c = {"X": bf(T, H), "dY": bf(T, H), "W1": bf(E, H, F).mul_(0.05), "W3": bf(E, H, F).mul_(0.05),
         "W2": bf(E, F, H).mul_(0.05), "k": k}
    z, idx = torch.topk(torch.randn(T, E, generator=g, device="cuda"), k, dim=1)
    c["w"] = torch.softmax(z, 1)
    _, c["offsets"], c["row_src"], c["assign_row"], _ = moe.permute(idx.int(), E)
    off = c["offsets"].tolist()
    Yp, ck = _forward(c)
    got = _backward(c, ck)
    # the last expert's last rows: forward
    e = max(i for i in range(E) if off[i + 1] > off[i])
    rows = torch.arange(max(off[e], off[e + 1] - 40), off[e + 1], device="cuda")
    token = lambda r: c["row_src"].long()[r] // k  # noqa: E731
    sub, part = _sub(c, ck, e, rows, token(rows))
    _check_forward(sub, Yp[rows], part)
    # the last tokens' gradients, over all their experts
    t = torch.arange(T - 12, T, device="cuda")
    r = torch.sort(c["assign_row"].long().reshape(T, k)[t].reshape(-1))[0]
    many = {n: c[n][t].cpu() for n in ("X", "dY", "w")} | {n: c[n].cpu() for n in ("W1", "W3", "W2")} | {
        "k": k, "row_src": (c["row_src"].long()[r] - (T - 12) * k).cpu().numpy(), "assign_row": None,
        "offsets": np.searchsorted(r.cpu().numpy(), np.array(off))} if k > 1 else None
    if many:
        _check_backward(many, moe.FFNCheckpoint(*(x[t] for x in ck[:2]), *(x[r] for x in ck[2:])),
                        (got[0][t], got[1][t], None, None, None))
    # the last expert's weight gradients, its last 32 columns of F
    rows = torch.arange(off[e], off[e + 1], device="cuda")
    sub, part = _sub(c, ck, e, rows, token(rows), slice(F - 32, F))
    _check_backward(sub, part, (None, None, got[2][e:e + 1, :, F - 32:], got[3][e:e + 1, :, F - 32:], got[4][e:e + 1, F - 32:]))


def test_ffn_train_nan_stays_in_its_expert():
    say("[train] a NaN row reaches its token and its expert only")
    c = _ffn_case(300, 64, 96, 6, 1)
    d = _dev(c)
    _, ck = _forward(d)
    clean = _backward(d, ck)
    t = 17
    r = int(c["assign_row"][t])
    e = int(np.searchsorted(c["offsets"], r, side="right") - 1)
    d["dY"] = d["dY"].clone()
    d["dY"][t, 5] = float("nan")
    got = _backward(d, ck)
    assert torch.isnan(got[0][t]).all() and torch.isnan(got[1][t]).all()
    rest = [i for i in range(300) if i != t]
    assert torch.equal(got[0][rest], clean[0][rest]) and torch.equal(got[1][rest], clean[1][rest])
    for a, b in zip(got[2:], clean[2:]):
        others = [i for i in range(6) if i != e]
        assert torch.equal(a[others], b[others]) and torch.isnan(a[e]).any()


def _step(d, X, dY, Wg, E, k, alpha, beta, seq):
    """One training step of the layer through the public calls."""
    logits, idx, w = moe.route(X, Wg, k)
    loss, counts, per = moe.balance_loss(logits, idx, alpha, beta, seq_offsets=seq)
    pc, off, src, inv, _ = moe.permute(idx, E)
    Yp, ck = moe.ffn_train_forward(X, off, d["W1"], d["W3"], d["W2"], row_src=src, k=k)
    Y = moe.combine(Yp, inv, w)
    dX, dw, dW1, dW3, dW2 = moe.ffn_train_backward(dY, ck, off, d["W1"], d["W3"], d["W2"], topk_w=w, row_src=src,
                                                   assign_row=inv)
    dz = moe.route_backward(logits, idx, w, dw, per, alpha, beta, seq_offsets=seq)
    return dict(logits=logits, idx=idx, w=w, loss=loss, counts=counts, pcounts=pc, off=off, src=src, inv=inv, Y=Y,
                Yp=Yp, ck=ck, dX=dX, dw=dw, dW1=dW1, dW3=dW3, dW2=dW2, dz=dz, per=per)


STEP = dict(T=150, H=96, F=160, E=8, k=2)


def _step_inputs(seed=0):
    c = _ffn_case(STEP["T"], STEP["H"], STEP["F"], STEP["E"], STEP["k"], seed=seed)
    g = torch.Generator().manual_seed(50 + seed)
    Wg = (0.3 * torch.randn(STEP["H"], STEP["E"], generator=g)).bfloat16()
    return c, Wg, torch.tensor([0, 40, 90, 150], dtype=torch.int32)


def test_training_step():
    say("[train] a whole step: route, losses, permute, FFN, combine and their gradients")
    c, Wg, seq = _step_inputs()
    d = _dev(c)
    o = _step(d, d["X"], d["dY"], Wg.cuda(), STEP["E"], STEP["k"], 0.02, 0.01, seq.cuda())
    assert torch.equal(o["counts"], o["pcounts"])
    c2 = dict(c) | {"w": o["w"].cpu(), "offsets": o["off"].cpu().numpy(), "row_src": o["src"].cpu().numpy(),
                    "assign_row": o["inv"].cpu().numpy()}
    _check_forward(c2, o["Yp"], o["ck"])
    _check_backward(c2, o["ck"], (o["dX"], o["dw"], o["dW1"], o["dW3"], o["dW2"]))
    _check_router(o["logits"].cpu(), o["idx"].cpu(), o["w"].cpu(), o["dw"].cpu(), seq.tolist(), 0.02, 0.01, (1.0, 1.0))
    # the inference path's rows: the same sums over H and F in another order
    # (its K splits differ), h and Yp rounded to bf16 by both
    ref = moe.grouped_ffn(d["X"], o["off"], d["W1"], d["W3"], d["W2"], row_src=o["src"], k=STEP["k"], path="tiled")
    _check_forward(c2, ref, o["ck"])


def test_training_step_graph_and_stream():
    say("[train] the step captured, replayed between eager work, on another stream, two at once")
    cases = [_step_inputs(s) for s in range(2)]
    (c, Wg, seq) = cases[0]
    d = _dev(c)
    X, dY, Wgd, sq = d["X"].clone(), d["dY"].clone(), Wg.cuda(), seq.cuda()
    names = ("Y", "dX", "dw", "dW1", "dW3", "dW2", "dz", "loss", "counts")
    run = lambda: _step(d, X, dY, Wgd, STEP["E"], STEP["k"], 0.02, 0.01, sq)  # noqa: E731
    eager = {}
    for i, (ci, _, _) in enumerate(cases):
        X.copy_(ci["X"])
        dY.copy_(ci["dY"])
        o = run()
        eager[i] = {n: o[n].clone() for n in names}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = run()
    for i in (0, 1, 0, 1, 1):
        X.copy_(cases[i][0]["X"])
        dY.copy_(cases[i][0]["dY"])
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(o[n], eager[i][n]), (i, n)
        run()  # eager work between the replays
        torch.cuda.synchronize()
    # two steps in flight on two streams
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, keep = [], []
    for i, s in enumerate(streams):
        Xi, dYi = cases[i][0]["X"].cuda(), cases[i][0]["dY"].cuda()
        keep.append((Xi, dYi))
    torch.cuda.synchronize()
    for (Xi, dYi), s in zip(keep, streams):
        with torch.cuda.stream(s):
            outs.append(_step(d, Xi, dYi, Wgd, STEP["E"], STEP["k"], 0.02, 0.01, sq))
    torch.cuda.synchronize()
    for i in range(2):
        for n in names:
            assert torch.equal(outs[i][n], eager[i][n]), (i, n)


def test_training_debug_build():
    say("[train] bounds-checked build: no failed check, the same bits")
    c, Wg, seq = _step_inputs()
    d = _dev(c)
    args = (d, d["X"], d["dY"], Wg.cuda(), STEP["E"], STEP["k"], 0.02, 0.01, seq.cuda())
    rel = _step(*args)
    torch.cuda.synchronize()
    dbg = _lib.load(_lib.DEBUG_LIB_PATH)
    with _lib.use_library(dbg):
        dbg.moe_debug_bounds()
        got = _step(*args)
        assert dbg.moe_debug_bounds() == 0
    for n in ("Y", "dX", "dw", "dW1", "dW3", "dW2", "dz", "loss"):
        assert torch.equal(rel[n], got[n]), n
