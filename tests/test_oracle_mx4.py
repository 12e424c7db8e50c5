"""CPU: the oracle of the 4-bit format and of the dispatch gradients against
hand-derived cases, other implementations, loops and differences."""
import numpy as np
import torch

import oracle
from oracle import dispatch, mx4
from synth.gen import quantize_mxfp4


def test_codes_of_every_value_and_tie():
    # a group whose largest magnitude is 6 has scale 1
    x = np.zeros((1, 32))
    x[0, :16] = [6, 0, .5, 1, 1.5, 2, 3, 4, -.5, -1, -1.5, -2, -3, -4, -6, -0.0]
    q, s = mx4.quantize_rows(x)
    assert s[0, 0] == 127
    np.testing.assert_array_equal(q[0, :8], [0x07, 0x21, 0x43, 0x65, 0xA9, 0xCB, 0xED, 0x8F])
    np.testing.assert_array_equal(mx4.row_values(q, s), x)
    # ties go to the even code: 0, 1, 1, 2, 2, 4, 4; past 6 to 6 (7.99 has the same scale)
    ties = np.zeros((1, 32))
    ties[0, :9] = [.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7.99, -5.01]
    np.testing.assert_array_equal(mx4.round_rows(ties)[0, :9], [0, 1, 1, 2, 2, 4, 4, 6, -6])


def test_scales():
    one = lambda v: mx4.quantize_rows(np.full((1, 32), v))[1][0, 0]  # noqa: E731
    assert one(0.0) == 127 and one(1.0) == 125 and one(-7.9) == 127 and one(8.0) == 128
    assert one(2.0 ** 127) == 252 and one(3.3e38) == 252
    assert one(2.0 ** -125) == 0 and one(2.0 ** -130) == 0      # at least 2^-127
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((2, 64))
        x[1, 40] = bad
        q, s = mx4.quantize_rows(x)
        np.testing.assert_array_equal(s, [[125, 125], [125, 255]])
        assert not q[1, 16:].any() and np.isnan(mx4.row_values(q, s)[1, 32:]).all()


def test_nearest_by_search():
    g = np.random.default_rng(1)
    x = g.standard_normal((40, 64)) * np.exp2(g.integers(-100, 100, (40, 1)))
    q, s = mx4.quantize_rows(x)
    v = mx4.row_values(q, s)
    scale = np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    grid = np.concatenate([-mx4.MAGS, mx4.MAGS])
    best = np.abs(x[:, :, None] / scale[:, :, None] - grid).min(axis=2)
    np.testing.assert_allclose(np.abs(x - v) / scale, best, rtol=1e-12, atol=1e-12)


def test_weights_as_the_synthetic_layers_store_them():
    g = torch.Generator().manual_seed(2)
    w = torch.randn(96, 40, generator=g) * torch.exp2(torch.randint(-30, 30, (1, 40), generator=g).float())
    w[32:64, 3] = 0.0
    q, s = mx4.quantize_weights(w.double().numpy())
    qr, sr = quantize_mxfp4(w)
    np.testing.assert_array_equal(s, sr.numpy())
    np.testing.assert_array_equal(mx4.weight_values(q, s), oracle.dequant_mxfp4(qr, sr))


def test_ffn_equals_swiglu_where_nothing_is_rounded():
    g = np.random.default_rng(3)
    x = g.choice([0.0, 1.0, -2.0], (5, 32))
    W1, W3 = np.eye(32)[:, :32] * 2, np.eye(32)
    y, gg, u, h, hq = mx4.ffn(x, W1, W3, np.eye(32))
    np.testing.assert_allclose(h, 2 * x / (1 + np.exp(-2 * x)) * x)
    np.testing.assert_array_equal(y, mx4.round_rows(h))
    np.testing.assert_array_equal(hq, y)


def _case(T, k, H, drop, seed):
    g = np.random.default_rng(seed)
    M = T * k
    a = g.permutation(M)
    n = M - drop
    return g.standard_normal((T, H)), g.standard_normal((M, H)), a, g.random((T, k)), n


def test_dispatch_gradients_by_loops_and_differences():
    for T, k, H, drop in ((4, 2, 3, 0), (5, 3, 4, 6), (1, 1, 2, 0)):
        dY, rows, a, w, n = _case(T, k, H, drop, T)
        dYp, dw = dispatch.combine_backward(dY, rows, a, w, n)
        dX = dispatch.permute_backward(rows, a, k, add=dY, n_rows=n)
        named = set()
        for t in range(T):
            want = dY[t].copy()
            for j in range(k):
                r = a[t * k + j]
                if r >= n:
                    assert dw[t, j] == 0
                    continue
                named.add(r)
                want += rows[r]
                np.testing.assert_allclose(dYp[r], w[t, j] * dY[t])
            np.testing.assert_allclose(dX[t], want)
        assert all(np.isnan(dYp[r]).all() for r in range(T * k) if r not in named)
        # differences of the sums that they are the gradients of

        def loss(Yp, wt):
            live = a < n
            return (wt.reshape(-1)[live, None] * Yp[a[live]] * dY[(np.arange(T * k) // k)[live]]).sum()
        eps = 1e-6
        for r in list(named)[:3]:
            for c in range(H):
                d = rows.copy()
                d[r, c] += eps
                assert abs((loss(d, w) - loss(rows, w)) / eps - dYp[r, c]) < 1e-6
        for t in range(T):
            d = w.copy()
            d[t, 0] += eps
            assert abs((loss(rows, d) - loss(rows, w)) / eps - dw[t, 0]) < 1e-6
