"""The oracle of the training operators against differences and closed forms
(CPU): gradients by central differences in fp64 of the forward's oracle, the
checkpoint format by its definition."""
import numpy as np
import pytest

import oracle
from oracle import train


def _differences(f, x, eps=1e-5):
    """Central differences of the scalar f at every element of x."""
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        v = x[i]
        x[i] = v + eps
        a = f()
        x[i] = v - eps
        d[i] = (a - f()) / (2 * eps)
        x[i] = v
    return d


def _case(T=9, E=6, k=2, seed=0):
    r = np.random.default_rng(seed)
    z = r.normal(size=(T, E))
    idx = oracle.select_topk(z, k)
    return r, z, idx


@pytest.mark.parametrize("seq", [None, [0, 9], [0, 4, 4, 9], [2, 5, 8]])
def test_route_backward_is_the_losses_gradient(seq):
    r, z, idx = _case()
    dl = (0.7, -1.3)

    def f():
        loss = train.balance_loss(z, idx, 0.3, 0.2, seq)[0]
        return dl[0] * loss[0] + dl[1] * loss[1]
    # truncation eps^2 |f'''| / 6 and rounding 1e-16 / eps: below 1e-9 here
    np.testing.assert_allclose(train.route_backward(z, idx, alpha=0.3, beta=0.2, seq=seq, dloss=dl),
                               _differences(f, z), atol=1e-9)


def test_route_backward_is_the_routing_weights_gradient():
    r, z, idx = _case(seed=1)
    dw = r.normal(size=idx.shape)
    got = train.route_backward(z, idx, oracle.routing_weights(z, idx), dw, aux=False)
    np.testing.assert_allclose(got, _differences(lambda: (oracle.routing_weights(z, idx) * dw).sum(), z), atol=1e-9)


def test_balance_loss_closed_forms():
    # uniform logits, every expert picked equally often: exactly alpha
    T, E, k = 12, 4, 2
    z = np.zeros((T, E))
    idx = np.array([[(t * k + j) % E for j in range(k)] for t in range(T)])
    loss, counts, per = train.balance_loss(z, idx, 0.5, 0.1, [0, 4, 12])
    assert abs(loss[0] - 0.5) < 1e-15 and abs(loss[1] - 0.1 * np.log(E) ** 2) < 1e-15
    assert counts.tolist() == [6] * E and per.tolist() == [[2] * E, [4] * E]
    # one expert takes everything, with certainty: alpha * E
    z[:, 1] = 800.0
    assert abs(train.balance_loss(z, np.ones((T, 1), dtype=int), 0.5, 0.0)[0][0] - 0.5 * E) < 1e-12
    # masked experts and masked rows
    z = np.full((3, 4), -np.inf)
    z[0, 2] = 1.0
    loss, _, _ = train.balance_loss(z, np.array([[2], [0], [0]]), 1.0, 1.0)
    assert abs(loss[1] - 1.0 / 3) < 1e-15 and np.isfinite(loss).all()
    assert np.isfinite(train.route_backward(z, np.array([[2], [0], [0]]), alpha=1.0, beta=1.0)).all()
    assert train.balance_loss(np.zeros((0, 4)), np.zeros((0, 2), dtype=int), 1.0, 1.0)[0].tolist() == [0.0, 0.0]


@pytest.mark.parametrize("k,seed", [(1, 0), (2, 1), (3, 2)])
def test_ffn_backward_is_the_forwards_gradient(k, seed):
    """Differences of <dY, combine(FFN)> in every input of the forward's oracle."""
    r = np.random.default_rng(seed)
    T, H, F, E = 5, 4, 3, 4
    X = r.normal(size=(T, H))
    W = {n: r.normal(size=s) for n, s in (("W1", (E, H, F)), ("W3", (E, H, F)), ("W2", (E, F, H)))}
    idx = np.stack([r.permutation(E)[:k] for _ in range(T)])
    w = r.uniform(0.2, 1.0, size=(T, k))
    dY = r.normal(size=(T, H))
    counts, offsets, row_src, assign_row = oracle.permute(idx, E)

    def f():
        Yp = oracle.grouped_ffn(X[row_src // k], offsets, lambda e: (W["W1"][e], W["W3"][e], W["W2"][e]))
        return (oracle.combine(Yp, assign_row, w, T, k) * dY).sum()
    e_of = np.repeat(np.arange(E), np.diff(offsets))
    xr = X[row_src // k]
    g = np.einsum("rh,rhf->rf", xr, W["W1"][e_of])
    u = np.einsum("rh,rhf->rf", xr, W["W3"][e_of])
    got = train.ffn_backward(dY, X, g, u, w, row_src, offsets, W["W1"], W["W3"], W["W2"], k)
    for name, x in (("dX", X), ("dw", w), ("dW1", W["W1"]), ("dW3", W["W3"]), ("dW2", W["W2"])):
        np.testing.assert_allclose(got[name], _differences(f, x), atol=2e-7, err_msg=name)


def test_checkpoint_format():
    r = np.random.default_rng(3)
    x = r.normal(size=(40, 96)) * np.exp2(r.integers(-140, 120, size=(40, 1)))
    x = np.clip(x, -3e38, 3e38)
    x[0] = 0.0
    q, s = train.checkpoint_pack(x)
    v = train.checkpoint_values(q, s)
    e = s.astype(np.float64) - 127
    top = np.abs(x.reshape(40, 3, 32)).max(axis=2)
    assert (top <= 448 * np.exp2(e)).all()
    assert ((top > 224 * np.exp2(e)) | (e == -126) | (top == 0)).all() and (e[0] == 0).all()
    # half a step: 2^-4 of the value, or half the smallest step 2^-9
    step = np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(np.exp2(e - 10), 32, axis=1))
    assert (np.abs(v - x) <= step).all()
    # exact at the format's edges: 448 fits its scale, the next number above takes the next
    x = np.zeros((3, 32))
    x[0, 5], x[1, 5], x[2, 5] = 448.0, np.nextafter(448.0, 1e9), 0.4375
    q, s = train.checkpoint_pack(x)
    assert s[:, 0].tolist() == [127, 128, 117] and q[0, 5] == 0x7e and q[2, 5] == 0x7e
    # values that are not finite become NaN and leave the scale alone
    x = np.ones((1, 32))
    x[0, 3], x[0, 4], x[0, 5] = np.nan, np.inf, -np.inf
    q, s = train.checkpoint_pack(x)
    v = train.checkpoint_values(q, s)
    assert np.isnan(v[0, 3:6]).all() and (v[0, 6:] == 1.0).all()
