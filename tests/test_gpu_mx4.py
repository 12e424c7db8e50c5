"""GPU: MXFP4 quantisation and the W4A4 expert FFN against the fp64 oracle
(oracle/mx4.py).

Codes and scales are compared bit for bit. The FFN's tolerance is a bound per
element, formed from the oracle's own terms: u = 2^-24 for each fp32 operation of a
sum (its length times u times the sum of magnitudes), half = 2^-8 for the output's
rounding to bf16, and, for each activation that lies within its own error of a
border between two codes, the distance of the two values times the weight."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_count_amd as moe
from mixture_experts_layer_count_amd import _lib
from oracle import mx4
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


# ----------------------------------------------------------------------------
# rows and weights
# ----------------------------------------------------------------------------
def _values(R, C, dt, seed, edges=True):
    """Rows of many sizes; with room for them, groups of zeros, of ties, of the largest
    and smallest numbers, and with NaN and infinities."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-120, 120, (R, 1), generator=g).float())
    if edges:
        ties = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -5, -.25, 7.9, -0.0, 0, .2500001, 4.999, 1e-30])
        special = [torch.zeros(16), ties, ties * 2.0 ** 40, ties * 2.0 ** -126, ties * 2.0 ** -130, torch.full((16,), 3.38e38),
                   torch.full((16,), 1e-44), torch.full((16,), 2.0 ** -124)]
        for i, v in enumerate(special):
            if i < R:
                x[i, :32] = v.repeat(2)
        for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
            if len(special) + i < R:
                x[len(special) + i, C - 5] = v
    return x.to(dt)


def _same_values(got, ref):
    """Equal, but for values below the smallest normal number, which may be flushed."""
    got, ref = np.array(got), np.array(ref)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    for v in (got, ref):
        v[np.abs(v) < 2.0 ** -126] = 0.0
    np.testing.assert_array_equal(got, ref)


@pytest.mark.parametrize("R,C,ld,dt", [(1, 32, 32, torch.bfloat16), (1, 32, 32, torch.float32),
                                       (13, 96, 104, torch.bfloat16), (12, 64, 68, torch.float32),
                                       (300, 2016, 2016, torch.bfloat16), (129, 7168, 7168, torch.bfloat16),
                                       (65, 1056, 1056, torch.float32)])
def test_rows_bit_exact(R, C, ld, dt):
    say(f"[mx4] rows {R} x {C} (rows of {ld}) {dt}")
    x = _values(R, ld, dt, R + C)
    X = x.cuda()[:, :C]
    Q, S = moe.quantize_mxfp4_rows(X)
    q, s = mx4.quantize_rows(f64(x[:, :C]))
    np.testing.assert_array_equal(S.cpu().numpy(), s)
    np.testing.assert_array_equal(Q.cpu().numpy(), q)
    for out in (torch.bfloat16, torch.float32):
        _same_values(f64(moe.dequantize_mxfp4_rows(Q, S, out)), mx4.row_values(q, s))


def test_rows_strided_and_empty():
    say("[mx4] a view with gaps between rows, one row, none")
    x = torch.randn(9, 3 * 160, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    view = x.view(9, 3, 160)[:, 1, :96]
    Q, S = moe.quantize_mxfp4_rows(view)
    q, s = moe.quantize_mxfp4_rows(view.contiguous())
    assert torch.equal(Q, q) and torch.equal(S, s)
    Q, S = moe.quantize_mxfp4_rows(view[4:5])
    assert torch.equal(Q, q[4:5]) and torch.equal(S, s[4:5])
    Q, S = moe.quantize_mxfp4_rows(x[:0])
    assert Q.shape == (0, 240) and S.shape == (0, 15) and moe.dequantize_mxfp4_rows(Q, S).shape == (0, 480)
    for bad in (x[:1].expand(9, 480), x.view(-1)[4:4 + 480].view(5, 96), x[:, :80]):
        with pytest.raises(moe.MoEError):  # rows on top of each other, off 16 bytes, no multiple of 32
            moe.quantize_mxfp4_rows(bad)


def test_every_code_and_scale():
    say("[mx4] every code under every scale")
    Q = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()           # 512 columns
    S = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 16).contiguous().cuda()
    ref = mx4.row_values(Q.cpu().numpy(), S.cpu().numpy())
    ref[np.abs(ref) >= 2.0 ** 128] *= np.inf        # past fp32's range
    _same_values(f64(moe.dequantize_mxfp4_rows(Q, S, torch.float32)), ref)
    W = moe.dequantize_mxfp4_weights(Q.T.contiguous(), S.T.contiguous(), torch.float32)
    assert torch.equal(W.T.nan_to_num(7), moe.dequantize_mxfp4_rows(Q, S, torch.float32).nan_to_num(7))


@pytest.mark.parametrize("G,K,N,dt", [(1, 32, 8, torch.bfloat16), (3, 64, 40, torch.float32), (8, 640, 416, torch.float32),
                                      (2, 1056, 2048, torch.bfloat16), (5, 96, 24, torch.bfloat16)])
def test_weights_bit_exact(G, K, N, dt):
    say(f"[mx4] weights {G} x {K} x {N} {dt}")
    w = torch.stack([_values(N, K, dt, G + K + i).T for i in range(G)]).contiguous()
    Q, S = moe.quantize_mxfp4_weights(w.cuda())
    back = {out: moe.dequantize_mxfp4_weights(Q, S, out) for out in (torch.bfloat16, torch.float32)}
    for e in range(G):
        q, s = mx4.quantize_weights(f64(w[e]))
        np.testing.assert_array_equal(S[e].cpu().numpy(), s)
        np.testing.assert_array_equal(Q[e].cpu().numpy(), q)
        for out, v in back.items():
            _same_values(f64(v[e]), mx4.weight_values(q, s))
    Q1, S1 = moe.quantize_mxfp4_weights(w[0].cuda())
    assert torch.equal(Q1, Q[0]) and torch.equal(S1, S[0])
    assert torch.equal(moe.dequantize_mxfp4_weights(Q1, S1).nan_to_num(7), back[torch.bfloat16][0].nan_to_num(7))


def test_past_32_bits():
    say("[mx4] rows and weights of more than 2^32 values")
    R, C = 70 * 1024, 65536
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    Q, S = moe.quantize_mxfp4_rows(x)
    q, s = moe.quantize_mxfp4_rows(x[-7:].clone())
    assert torch.equal(Q[-7:], q) and torch.equal(S[-7:], s)
    assert torch.equal(moe.dequantize_mxfp4_rows(Q, S)[-7:], moe.dequantize_mxfp4_rows(q, s))
    w = x.view(70, 1024, C)
    Q, S = moe.quantize_mxfp4_weights(w)
    q, s = moe.quantize_mxfp4_weights(w[-1].clone())
    assert torch.equal(Q[-1], q) and torch.equal(S[-1], s)
    assert torch.equal(moe.dequantize_mxfp4_weights(Q, S)[-1], moe.dequantize_mxfp4_weights(q, s))


# ----------------------------------------------------------------------------
# the expert FFN
# ----------------------------------------------------------------------------
def _experts(E, H, F, seed, scale=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = {}
    for n, s in (("W1", (E, H, F)), ("W3", (E, H, F)), ("W2", (E, F, H))):
        d[n], d["S" + n[1]] = moe.quantize_mxfp4_weights(scale * torch.randn(*s, generator=g, device="cuda"))
    return d


def _case(T, H, F, E, k, seed, lean=0.0, scale=0.05):
    """Experts, tokens and a permutation; `lean` makes the first experts popular and
    leaves the last ones without rows."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) - lean * torch.arange(E)
    idx = torch.topk(z, k, dim=1)[1].int().cuda()
    _, off, src, back, _ = moe.permute(idx, E)
    x = torch.randn(T, H, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    return _experts(E, H, F, seed, scale) | {"X": x.bfloat16().cuda(), "offsets": off, "row_src": src, "assign_row": back,
                                             "idx": idx, "k": k, "E": E}


def _ffn(d, **kw):
    return moe.grouped_ffn(d["X"], d["offsets"], d["W1"], d["W3"], d["W2"], d["S1"], d["S3"], d["S2"],
                           **{"row_src": d["row_src"], "k": d["k"], "path": "tiled_a4"} | kw)


def _bounded(xe, W1, W3, W2):
    """The exact output of one expert's rows and its bound per element."""
    xq = mx4.round_rows(xe)
    y, g, u, h, hq = mx4.ffn(xq, W1, W3, W2)
    H, F = W1.shape
    dg, du = ((H + 8) * U * (np.abs(xq) @ np.abs(W)) for W in (W1, W3))
    with np.errstate(over="ignore"):
        silu = np.abs(g / (1 + np.exp(-g)))
    dh = 1.1 * dg * np.abs(u) + (silu + 1.1 * dg) * du + 10 * U * np.abs(h)
    # activations that may fall on the other side of a border between codes
    grp = lambda v: v.reshape(v.shape[0], -1, 32)  # noqa: E731
    amax, err = np.abs(grp(h)).max(axis=2), grp(dh).max(axis=2)
    e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1))) - 2, 0)
    s = np.repeat(np.exp2(np.maximum(e, -127)), 32, axis=1)
    dev = np.zeros_like(h)
    for i in range(7):
        border = (mx4.MAGS[i] + mx4.MAGS[i + 1]) / 2 * s
        dev = np.where(np.abs(np.abs(h) - border) <= dh, (mx4.MAGS[i + 1] - mx4.MAGS[i]) * s, dev)
    # and groups whose largest magnitude may have the next power of two: one rounding
    # step of either scale, and what saturates under the smaller
    with np.errstate(divide="ignore"):
        moved = np.floor(np.log2(amax + err)) != np.floor(np.log2(np.maximum(amax - err, 1e-300)))
    dev = np.where(np.repeat(moved & (amax > 0), 32, axis=1), 6 * s, dev)
    tol = (F + 8) * U * ((np.abs(hq) + dev) @ np.abs(W2)) + dev @ np.abs(W2)
    return y, tol + HALF * (np.abs(y) + tol) + 2.0 ** -133


def _check(d, Y, rows=None):
    """Y against the oracle, on all rows in use or on some of them."""
    off, src, x = d["offsets"].tolist(), d["row_src"].long().cpu().numpy(), f64(d["X"])
    worst = 0.0
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        r = np.arange(lo, hi) if rows is None else np.array([v for v in rows if lo <= v < hi], dtype=int)
        if not r.size:
            continue
        W = [mx4.weight_values(d[n][e].cpu().numpy(), d["S" + n[1]][e].cpu().numpy()) for n in ("W1", "W3", "W2")]
        y, tol = _bounded(x[src[r] // d["k"]], *W)
        off_by = np.abs(f64(Y[torch.as_tensor(r, device="cuda")]) - y)
        assert (off_by <= tol).all(), f"expert {e}: {(off_by > tol).sum()} of {y.size} out, worst {np.nanmax(off_by / tol):.3g} of the bound"
        worst = max(worst, float((off_by / tol).max()))
    say(f"    worst {worst:.2f} of the bound")


# rows an expert: one; fewer than any tile's; a tile's and one more or less; several tiles of each height
@pytest.mark.parametrize("T,H,F,E,k", [(1, 32, 32, 1, 1), (1, 128, 256, 8, 2), (3, 96, 160, 4, 3), (64, 160, 96, 1, 1),
                                       (65, 256, 32, 1, 1), (300, 640, 416, 8, 2), (191, 352, 288, 1, 1),
                                       (193, 128, 128, 1, 1), (257, 2080, 224, 1, 1), (513, 512, 1056, 2, 1),
                                       (700, 1024, 384, 3, 2), (1500, 288, 768, 16, 3), (2100, 64, 2112, 5, 4)])
def test_ffn(T, H, F, E, k):
    say(f"[mx4] ffn T={T} H={H} F={F} E={E} k={k}")
    d = _case(T, H, F, E, k, T + H)
    Y = _ffn(d)
    assert torch.equal(Y, _ffn(d))
    _check(d, Y)
    # the same rows, gathered beforehand
    Xp = d["X"][d["row_src"].long() // k].contiguous()
    assert torch.equal(Y, _ffn(d | {"X": Xp, "k": 1}, row_src=None))


@pytest.mark.parametrize("T,H,F,E,k,lean", [(900, 256, 320, 12, 2, 0.6), (4096, 128, 128, 64, 1, 0.2), (33, 64, 96, 32, 2, 0.0)])
def test_ffn_uneven_and_empty_experts(T, H, F, E, k, lean):
    say(f"[mx4] ffn with uneven experts T={T} E={E} k={k}")
    d = _case(T, H, F, E, k, T, lean)
    n = (d["offsets"][1:] - d["offsets"][:-1]).tolist()
    say(f"    rows {sorted(n)}")
    assert min(n) == 0 or lean == 0.2
    _check(d, _ffn(d))


@pytest.mark.parametrize("T,H,F,E", [(40, 7168, 64, 1),       # one tile a product: parts over K
                                     (300, 3584, 3200, 1),    # fewer tiles than compute units
                                     (1100, 1536, 1568, 8)])  # more, the last round in parts
def test_ffn_in_parts_over_k(T, H, F, E):
    say(f"[mx4] ffn whose tiles are cut over K: T={T} H={H} F={F} E={E}")
    d = _case(T, H, F, E, 1, T)
    Y = _ffn(d)
    for _ in range(3):
        assert torch.equal(Y, _ffn(d))  # whichever part is last
    _check(d, Y, rows=range(0, T, max(1, T // 60)))


def test_ffn_many_tiles_a_workgroup():
    say("[mx4] ffn of more tiles than one round's tables hold")
    T, H, F, E = 2000, 64, 4096, 1024
    d = _case(T, H, F, E, 2, 5)
    Y = _ffn(d)
    _check(d, Y, rows=list(range(0, 40)) + list(range(4000 - 40, 4000)))


def test_ffn_rows_behind_the_last_group():
    say("[mx4] ffn whose last rows belong to no expert")
    d = _case(200, 96, 64, 4, 2, 9)
    off = d["offsets"].clone()
    full = _ffn(d)
    cut = int(off[3])
    off[4] = cut                     # the last expert's rows are left out
    src = d["row_src"].clone()
    src[cut:] = 0x7ffffff0           # never read
    out = torch.full((400, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    _ffn(d | {"offsets": off, "row_src": src}, out=out)
    assert torch.equal(out[:cut], full[:cut]) and (out[cut:] == 7).all()
    _ffn(d | {"offsets": torch.zeros_like(off)}, out=out.fill_(3.0))
    assert (out == 3).all()


def test_ffn_rows_of_any_assignments():
    """Many rows whose assignments are no permutation: one twice, some missing, some past
    the number of rows (other ranks' tokens)."""
    say("[mx4] ffn of many rows, some of the same assignment, some past the rows' number")
    T, H, F, E, k = 16000, 1056, 64, 6, 4
    d = _case(T, H, F, E, k, 15)
    src = d["row_src"].clone()
    g = torch.Generator().manual_seed(4)
    at = torch.randperm(T * k, generator=g)[:700].cuda()
    src[at[:300]] = src[at[300:600]]                        # twice
    M = 60001                                               # fewer rows than assignments
    off = d["offsets"].clamp(max=M)
    src = src[:M].clone()
    assert int((src >= M).sum()) > 500 and src.unique().numel() < M
    Y = _ffn(d | {"row_src": src, "offsets": off})
    Xp = d["X"][src.long() // k].contiguous()
    assert torch.equal(Y, _ffn(d | {"X": Xp, "k": 1, "offsets": off}, row_src=None))
    _check(d | {"row_src": src, "offsets": off}, Y, rows=range(0, M, 797))
    # no rows in use, nothing read
    out = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
    _ffn(d | {"row_src": torch.full_like(src, 0x7ffffff0), "offsets": torch.zeros_like(off)}, out=out)
    assert (out == 7).all()


@pytest.mark.parametrize("k", [5, 64, 65, 60000, 2**31 - 1])
def test_ffn_rows_of_any_picks_a_token(k):
    say(f"[mx4] ffn of many rows, {k} picks a token")
    M, H = 60000, 1056
    d = _experts(3, H, 32, 7)
    g = torch.Generator(device="cuda").manual_seed(k % 1000)
    src = torch.randint(0, min(2**31 - 1, 20 * k), (M,), generator=g, device="cuda", dtype=torch.int64)
    x = torch.randn(int(src.max()) // k + 1, H, generator=g, device="cuda").bfloat16()
    d |= {"X": x, "offsets": torch.tensor([0, 20000, 20001, M], dtype=torch.int32, device="cuda"), "k": k}
    y = _ffn(d | {"row_src": src.int()})
    assert torch.equal(y, _ffn(d | {"X": x[src // k].contiguous(), "k": 1, "row_src": None}))


# tiles of 256, 256, 192, 128 rows, more than one round of them and a part of one (in whole
# tiles or in pieces of 64 rows, some without rows), for gate/up (wide F) or down (wide H)
@pytest.mark.parametrize("sizes", [[700, 257, 64, 1000, 579], [1, 2598, 1, 0], [6, 300, 64, 65, 128, 193, 0, 192, 1, 250] * 2,
                                   [7, 64, 65, 130, 0, 1, 127, 128, 129, 10] * 3], ids=["tall", "lone", "mid", "short"])
@pytest.mark.parametrize("H,F", [(96, 2944), (5888, 64), (96, 1504), (3040, 128)])
def test_ffn_of_all_experts_is_that_of_each(sizes, H, F):
    """A row's sums run over K in one order, whatever tile or piece it lies in."""
    say(f"[mx4] ffn of {len(sizes)} experts, together and one by one, H={H} F={F}")
    E, M = len(sizes), sum(sizes)
    d = _experts(E, H, F, M + H)
    g = torch.Generator(device="cuda").manual_seed(F)
    x = torch.randn(M, H, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    names = ("W1", "W3", "W2", "S1", "S3", "S2")
    run = lambda: moe.grouped_ffn(x, off, *(d[n] for n in names), path="tiled_a4")  # noqa: E731
    y = run()
    at = 0
    for e, n in enumerate(sizes):
        if n:
            one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            ye = moe.grouped_ffn(x[at:at + n], one, *(d[m][e:e + 1] for m in names), path="tiled_a4")
            assert torch.equal(y[at:at + n], ye), e
        at += n
    h = _lib.load(_lib.DEBUG_LIB_PATH)
    h.moe_debug_bounds()
    with _lib.use_library(h):
        assert torch.equal(run(), y) and h.moe_debug_bounds() == 0


def test_ffn_nan_and_infinity_stay_in_their_rows():
    say("[mx4] ffn with NaN, infinity and the NaN scale")
    d = _case(150, 256, 160, 3, 1, 11)
    clean = _ffn(d)
    x = d["X"].clone()
    x[5, 40], x[77, 200], x[149, 0] = float("nan"), float("inf"), -float("inf")
    Y = _ffn(d | {"X": x})
    rows = d["assign_row"].long()
    bad = torch.zeros(150, dtype=torch.bool, device="cuda")
    bad[rows[torch.tensor([5, 77, 149])]] = True
    assert torch.isnan(Y[bad]).all() and torch.equal(Y[~bad], clean[~bad])
    # a weight column whose scale is NaN
    s2 = d["S2"].clone()
    s2[1, 2, 17] = 255
    Y = _ffn(d | {"S2": s2})
    lo, hi = d["offsets"][1].item(), d["offsets"][2].item()
    assert torch.isnan(Y[lo:hi, 17]).all()
    Y[lo:hi, 17] = clean[lo:hi, 17]
    assert torch.equal(Y, clean)


def test_ffn_small_and_large_scales():
    say("[mx4] ffn at the ends of the scales' range")
    d = _case(70, 64, 64, 2, 1, 13)
    x = torch.zeros(70, 64)
    x[:, ::3] = 2.0 ** -126                       # scale byte 0 or 1
    big = {n: torch.full_like(d[n], 250) for n in ("S1", "S3")}
    dd = d | {"X": x.bfloat16().cuda(), "S1": big["S1"] - 25, "S3": big["S3"] - 25}
    _check(dd, _ffn(dd))
    dd = d | {"X": (x.double() * 2.0 ** 200).bfloat16().cuda(), "S1": torch.full_like(d["S1"], 30), "S3": torch.full_like(d["S3"], 60)}
    _check(dd, _ffn(dd))


def test_ffn_past_32_bits():
    say("[mx4] ffn whose panels and outputs pass 2^32 bytes")
    M, H, F = (1 << 20) + 77, 8192, 128
    g = torch.Generator(device="cuda").manual_seed(17)
    d = _experts(2, H, F, 17) | {"k": 1, "E": 2}
    d["X"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    d["offsets"] = torch.tensor([0, 1000, M], dtype=torch.int32, device="cuda")
    d["row_src"] = torch.arange(M, dtype=torch.int32, device="cuda")
    Y = _ffn(d, row_src=None)
    r = [0, 999, 1000, M // 2, M - 2, M - 1]
    sub = d | {"X": d["X"][r].contiguous(), "offsets": torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda"),
               "row_src": torch.arange(6, dtype=torch.int32, device="cuda")}
    _check(sub, Y[r])
    del Y
    Yg = _ffn(d)                                  # gathered
    _check(sub, Yg[r])


def test_ffn_refusals():
    d = _case(40, 64, 96, 3, 2, 3)
    for bad in ({"S1": d["S1"][:, :1]}, {"S2": d["S2"].transpose(1, 2).contiguous()}, {"W3": d["W3"][:2]},
                {"offsets": d["offsets"][:3]}, {"row_src": d["row_src"][:5]}):
        with pytest.raises(ValueError):
            _ffn(d | bad, M=80)
    with pytest.raises(TypeError):
        _ffn(d | {"S3": d["S3"].float()})
    with pytest.raises(moe.MoEError):
        moe.grouped_ffn(d["X"], d["offsets"], *(torch.zeros(s, dtype=torch.bfloat16, device="cuda")
                                                for s in ((3, 64, 96), (3, 64, 96), (3, 96, 64))), path="tiled_a4",
                        row_src=d["row_src"], k=2)


# ----------------------------------------------------------------------------
# the layer
# ----------------------------------------------------------------------------
def _layer(T, H, F, E, k, Fs, shared, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = _experts(E, H, F, seed)
    d["Wg"] = (0.05 * torch.randn(H, E, generator=g, device="cuda")).bfloat16()
    d["X"] = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    for n, s in (("Ws1", (H, Fs)), ("Ws3", (H, Fs)), ("Ws2", (Fs, H))):
        w = 0.05 * torch.randn(*s, generator=g, device="cuda") if Fs else None
        if shared == "mxfp4":
            d[n], d["S" + n[1:]] = moe.quantize_mxfp4_weights(w)
        elif shared:
            d[n] = w.bfloat16()
    return d


@pytest.mark.parametrize("T,H,F,E,k,Fs,shared", [(1, 256, 128, 8, 2, 0, None), (130, 384, 160, 8, 3, 160, "mxfp4"),
                                                 (700, 256, 416, 16, 4, 96, "bf16"), (2500, 512, 256, 4, 1, 256, "mxfp4"),
                                                 (3300, 1088, 64, 12, 5, 64, "mxfp4")])
def test_layer_is_its_stages(T, H, F, E, k, Fs, shared):
    say(f"[mx4] layer T={T} H={H} F={F} E={E} k={k} shared {shared}")
    d = _layer(T, H, F, E, k, Fs, shared, T)
    layer = moe.MoELayer(d, k, path="tiled_a4")
    Y, logits, idx, w, counts = layer.forward(d["X"], aux=True)
    assert torch.equal(Y, layer.forward_noalloc(d["X"]))
    _, off, src, back, _ = moe.permute(idx, E)
    Yp = _ffn(d | {"offsets": off, "row_src": src, "k": k})
    S = None
    if Fs:
        one = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        ws = [d[n].unsqueeze(0) for n in ("Ws1", "Ws3", "Ws2")]
        if shared == "mxfp4":
            S = moe.grouped_ffn(d["X"], one, *ws, *(d[n].unsqueeze(0) for n in ("Ss1", "Ss3", "Ss2")), path="tiled_a4")
        else:
            S = moe.grouped_ffn(d["X"], one, *ws, path="tiled")
    want = moe.combine(Yp, back, w, S)
    # fp32 sums of tiles of another height or cut into other parts round apart by a bf16 step of a term at most
    terms = (w.unsqueeze(2) * Yp[back.long()].float().view(T, k, H).abs()).sum(1) + (0 if S is None else S.float().abs())
    assert ((Y.float() - want.float()).abs() <= 4 * HALF * terms + 1e-30).all()


def test_layer_over_ranks():
    say("[mx4] layer with its experts over 4 ranks of one device")
    d = _layer(160, 256, 128, 16, 3, 128, "mxfp4", 7)
    Y = moe.MoELayer(d, 3, path="tiled_a4").forward(d["X"])
    Ye = moe.EPLoopback(d, 3, 4, path="tiled_a4").forward(d["X"])
    assert (Y.float() - Ye.float()).abs().max() <= 4 * HALF * Y.float().abs().max()


# ----------------------------------------------------------------------------
# graphs, streams, the bounds-checked build
# ----------------------------------------------------------------------------
def _all(d, W):
    """Every 4-bit operator once; outputs in a list."""
    Q, S = moe.quantize_mxfp4_rows(d["X"])
    WQ, WS = moe.quantize_mxfp4_weights(W)
    return [Q, S, moe.dequantize_mxfp4_rows(Q, S), WQ, WS, moe.dequantize_mxfp4_weights(WQ, WS), _ffn(d)]


def test_captured_and_replayed():
    say("[mx4] captured, replayed with other inputs and eager work between")
    d = _case(500, 1600, 224, 4, 2, 21)             # 13 steps: tiles in parts too
    W = torch.randn(2, 64, 48, device="cuda")
    _all(d, W)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _all(d, W)
    for seed in range(4):
        d["X"].copy_(torch.randn(500, 1600, generator=torch.Generator().manual_seed(seed)))
        W.copy_(torch.randn(2, 64, 48, generator=torch.Generator().manual_seed(seed)))
        want = _all(d, W)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        torch.randn(1 << 20, device="cuda").sum().item()


def test_two_streams():
    say("[mx4] two streams at once")
    cases = [_case(600, 1600, 160, 4, 2, 31), _case(333, 96, 2080, 3, 1, 32)]
    want = [_ffn(d) for d in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, (s, d) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                got[i].append(_ffn(d))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(v, w) for v in g)


def test_bounds_checked_build():
    say("[mx4] the bounds-checked build")
    cases = [_case(300, 640, 416, 8, 2, 41), _case(2100, 64, 2112, 5, 4, 42), _case(40, 7168, 64, 1, 1, 43),
             _case(1, 32, 32, 1, 1, 44)]
    d = _layer(300, 384, 160, 8, 3, 160, "mxfp4", 45)
    run = lambda: [_ffn(c) for c in cases] + [moe.MoELayer(d, 3, path="tiled_a4").forward(d["X"])]  # noqa: E731
    want = run()
    h = _lib.load(_lib.DEBUG_LIB_PATH)
    h.moe_debug_bounds()
    with _lib.use_library(h):
        got = run()
        assert h.moe_debug_bounds() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
