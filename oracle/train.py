"""fp64 oracle of the layer's training operators: router losses and the
gradient at the logits, 8-bit activation checkpoints, and the backward pass of
the grouped FFN. Formulas as include/moe.h states them; pinned by differences
of the forward's oracle (tests/test_oracle_train.py)."""
from __future__ import annotations

import numpy as np

from .ref import _e4m3_table, e4m3_encode, silu, softmax


def _sequences(T, seq):
    """(first, last + 1) of every sequence."""
    seq = [0, T] if seq is None else [int(v) for v in np.asarray(seq)]
    return list(zip(seq, seq[1:]))


def log_sum_exp(logits) -> np.ndarray:
    z = np.asarray(logits, dtype=np.float64)
    top = z.max(axis=1)
    base = np.where(np.isneginf(top), 0.0, top)
    with np.errstate(divide="ignore"):
        lse = base + np.log(np.exp(z - base[:, None]).sum(axis=1))
    return np.where(np.isneginf(top), 0.0, lse)


def probabilities(logits) -> np.ndarray:
    """softmax; 0 for a row of -inf only."""
    z = np.asarray(logits, dtype=np.float64)
    dead = np.isneginf(z.max(axis=1))
    return np.where(dead[:, None], 0.0, softmax(np.where(dead[:, None], 0.0, z)))


def _fractions(idx, E, seqs):
    k = idx.shape[1]
    counts = np.zeros((len(seqs), E), dtype=np.int64)
    for b, (lo, hi) in enumerate(seqs):
        e = idx[lo:hi].reshape(-1)
        counts[b] = np.bincount(e[(e >= 0) & (e < E)], minlength=E)
    n = np.array([hi - lo for lo, hi in seqs], dtype=np.float64)
    return counts, E * counts / (k * np.maximum(n, 1.0))[:, None], n


def balance_loss(logits, idx, alpha, beta, seq=None):
    """-> (loss [2], counts [E], seq_counts [B,E])."""
    z, idx = np.asarray(logits, dtype=np.float64), np.asarray(idx)
    T, E = z.shape
    seqs = _sequences(T, seq)
    counts, f, n = _fractions(idx, E, seqs)
    p, lse = probabilities(z), log_sum_exp(z)
    live, N = (n > 0).sum(), n.sum()
    bal = sum((f[b] * p[lo:hi].mean(axis=0)).sum() for b, (lo, hi) in enumerate(seqs) if hi > lo)
    zz = sum((lse[lo:hi] ** 2).sum() for lo, hi in seqs)
    loss = np.array([alpha * bal / live if live else 0.0, beta * zz / N if N else 0.0])
    return loss, counts.sum(axis=0), counts


def route_backward(logits, idx, w=None, dw=None, alpha=0.0, beta=0.0, seq=None, dloss=(1.0, 1.0), aux=True):
    """dlogits [T,E]; aux: the two losses' terms, w and dw: the routing weights'."""
    z, idx = np.asarray(logits, dtype=np.float64), np.asarray(idx)
    T, E = z.shape
    d = np.zeros((T, E))
    if aux:
        seqs = _sequences(T, seq)
        _, f, n = _fractions(idx, E, seqs)
        p, lse = probabilities(z), log_sum_exp(z)
        live, N = (n > 0).sum(), n.sum()
        for b, (lo, hi) in enumerate(seqs):
            if hi <= lo:
                continue
            q = p[lo:hi]
            d[lo:hi] += dloss[0] * alpha / (live * n[b]) * q * (f[b] - (q * f[b]).sum(axis=1, keepdims=True))
            d[lo:hi] += dloss[1] * 2 * beta / N * lse[lo:hi, None] * q
    if dw is not None:
        w, dw = np.asarray(w, dtype=np.float64), np.asarray(dw, dtype=np.float64)
        v = w * (dw - (w * dw).sum(axis=1, keepdims=True))
        for t in range(T):
            for j in range(idx.shape[1]):
                if 0 <= idx[t, j] < E:
                    d[t, idx[t, j]] += v[t, j]
    return d


def checkpoint_scales(x) -> np.ndarray:
    """Scale exponents [R, C/32]: the smallest e in [-126, 127] with the group's
    largest finite magnitude <= 448 * 2^e; 0 for a group of zeros."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x.reshape(x.shape[0], -1, 32))
    top = np.where(np.isfinite(a), a, 0.0).max(axis=2)
    e = np.full(top.shape, -126, dtype=np.int64)
    for step in (128, 64, 32, 16, 8, 4, 2, 1):       # largest e' with 448 * 2^e' < amax, then one more
        more = (448.0 * np.exp2((e + step - 1).astype(np.float64)) < top) & (e + step <= 127)
        e = np.where(more, e + step, e)
    return np.where(top == 0.0, 0, e)


def checkpoint_pack(x):
    """-> (codes uint8 [R,C], scale bytes uint8 [R,C/32])."""
    x = np.asarray(x, dtype=np.float64)
    e = checkpoint_scales(x)
    v = x.reshape(x.shape[0], -1, 32) * np.exp2(-e.astype(np.float64))[:, :, None]
    q = e4m3_encode(np.where(np.isfinite(v), v, np.nan)).reshape(x.shape)
    return q, (e + 127).astype(np.uint8)


def checkpoint_values(q, s) -> np.ndarray:
    q, s = np.asarray(q, dtype=np.uint8), np.asarray(s, dtype=np.float64)
    v = _e4m3_table()[q].reshape(q.shape[0], -1, 32)
    return (v * np.exp2(s - 127)[:, :, None]).reshape(q.shape)


def swiglu_backward(g, u):
    """(h, dh/du = g s, dh/dg) at the projections g, u."""
    s = 1.0 / (1.0 + np.exp(-g))
    return silu(g) * u, g * s, u * s * (1.0 + g * (1.0 - s))


def ffn_backward(dY, x, g, u, w, row_src, offsets, W1, W3, W2, k):
    """Backward of the grouped FFN and combine from token rows x [T,H], the
    projections g, u [M,F] and routing weights w [T,k] (None: 1). Returns a dict
    with dX, dw, dW1, dW3, dW2 and, for error bounds, p, dg, du, h by row. `row_src`
    None: row r is token r."""
    dY, x, g, u = (np.asarray(v, dtype=np.float64) for v in (dY, x, g, u))
    T, H = dY.shape
    M, F = g.shape
    src = np.arange(M) if row_src is None else np.asarray(row_src)
    wr = np.ones(M) if w is None else np.asarray(w, dtype=np.float64).reshape(-1)[src]
    G = len(offsets) - 1
    h, hu, hg = swiglu_backward(g, u)
    out = {"dX": np.zeros((T, H)), "dw": np.zeros(T * k), "dW1": np.zeros((G, H, F)), "dW3": np.zeros((G, H, F)),
           "dW2": np.zeros((G, F, H)), "p": np.zeros((M, F)), "h": h, "hu": hu, "hg": hg, "w": wr, "src": src}
    for e in range(G):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        t = src[lo:hi] // k
        w1, w3, w2 = (np.asarray(v[e], dtype=np.float64) for v in (W1, W3, W2))
        p = dY[t] @ w2.T
        out["p"][lo:hi] = p
        out["dw"][src[lo:hi]] = (p * h[lo:hi]).sum(axis=1)
        wp = wr[lo:hi, None] * p
        dg, du = wp * hg[lo:hi], wp * hu[lo:hi]
        np.add.at(out["dX"], t, dg @ w1.T + du @ w3.T)
        out["dW1"][e], out["dW3"][e] = x[t].T @ dg, x[t].T @ du
        out["dW2"][e] = (wr[lo:hi, None] * h[lo:hi]).T @ dY[t]
    out["dw"] = out["dw"].reshape(T, k)
    return out
