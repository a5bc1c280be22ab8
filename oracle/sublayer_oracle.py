"""Plain fp64 CPU oracle of the experts' forward, its backward, layer norm and dropout.

TEST INFRASTRUCTURE ONLY, like ``lrm_oracle``: written from the formulas, with
none of the CUDA library's code.
"""

from __future__ import annotations

import numpy as np

__all__ = ["ffn_up", "ffn_down", "ffn_combine", "ffn_backward", "layer_norm", "layer_norm_backward", "philox4x32_10",
           "dropout_kept"]


def _silu(a):
    with np.errstate(over="ignore"):
        return a / (1.0 + np.exp(-a))


def _silu_grad(a):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-a))
    return s + a * s * (1.0 - s)


def ffn_up(x, W1, offsets, ids, k):
    """[a | b] and silu(a) b of the pairs of every segment, by segment row."""
    I = W1.shape[1] // 2
    ab = np.zeros((len(ids), 2 * I))
    for e in range(W1.shape[0]):
        seg = slice(offsets[e], offsets[e + 1])
        ab[seg] = x[ids[seg] // k] @ W1[e].T
    return ab, _silu(ab[:, :I]) * ab[:, I:]


def ffn_down(phi, W, offsets, ids):
    """W_e phi[u] of the pairs of every segment, by segment row."""
    out = np.zeros((len(ids), W.shape[1]))
    for e in range(W.shape[0]):
        seg = slice(offsets[e], offsets[e + 1])
        out[seg] = phi[ids[seg]] @ W[e].T
    return out


def ffn_combine(rows, alpha, k):
    """sum over a token's pairs of alpha row, pairs with gate 0 left out."""
    T = len(alpha) // k
    used = np.where((alpha != 0)[:, None], rows, 0.0)
    return (alpha[:, None] * used).reshape(T, k, -1).sum(1)


def ffn_backward(delta, W, ab, offsets, ids, N):
    """[dphi b silu'(a) | dphi silu(a)] by segment row, and <dphi, silu(a) b> by pair."""
    I = W.shape[2]
    dphi = np.zeros((len(ids), I))
    for e in range(W.shape[0]):
        seg = slice(offsets[e], offsets[e + 1])
        dphi[seg] = delta[seg] @ W[e]
    a, b = ab[ids, :I], ab[ids, I:]
    dgate = np.zeros(N)
    dgate[ids] = (dphi * _silu(a) * b).sum(1)
    return np.concatenate([dphi * b * _silu_grad(a), dphi * _silu(a)], 1), dgate


def layer_norm(x, gamma, beta, eps, valid=None):
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * gamma + beta
    stats = np.stack([mean, rstd], 1)
    if valid is not None:
        y, stats = np.where(valid[:, None] != 0, y, 0.0), np.where(valid[:, None] != 0, stats, 0.0)
    return y, stats


def layer_norm_backward(x, dy, gamma, stats, valid=None, dres=None):
    keep = np.ones(len(x), bool) if valid is None else valid != 0
    xhat = (x[keep] - stats[keep, :1]) * stats[keep, 1:]
    d = dy[keep] * gamma
    dx = np.zeros_like(x)
    dx[keep] = stats[keep, 1:] * (d - d.mean(1, keepdims=True) - xhat * (d * xhat).mean(1, keepdims=True))
    if dres is not None:
        dx[keep] += dres[keep]
    return dx, (dy[keep] * xhat).sum(0), dy[keep].sum(0)


def philox4x32_10(counter, key):
    """Philox4x32-10 (Salmon et al., SC 2011, sec. 3.2) of counters [n, 4] under a key of two words."""
    c = np.asarray(counter, dtype=np.uint64).T.copy()
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = np.stack([(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & low,
                      (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & low])
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c.T


def dropout_kept(n, p, seed, offset, first=0):
    """Which of the elements first .. first + n - 1 dropout keeps."""
    q = np.arange(first // 4, (first + n + 3) // 4, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    offset &= (1 << 64) - 1
    counter = np.stack([q & low, q >> np.uint64(32), np.full_like(q, offset & 0xFFFFFFFF),
                        np.full_like(q, offset >> 32)], 1)
    words = philox4x32_10(counter, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)).reshape(-1)
    return words[first % 4:first % 4 + n] >= int(np.floor(p * 2.0 ** 32))
