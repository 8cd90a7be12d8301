"""Plain 64-bit forms of the norm, the gated activation and the router with
scores, a bias and groups, for their tests: numpy, written from the definitions
in include/q4.h. Pinned by test_plain_rows.py."""
import math

import numpy as np

from plain_experts import bf16_value


def widen(x):
    """f32 values, or bfloat16 patterns (uint16), in f64."""
    x = np.asarray(x)
    return (bf16_value(x) if x.dtype == np.uint16 else x).astype(np.float64)


def norm_sum(x, weights, share, residual):
    """(h, the sum of its terms' sizes), [M, K] in f64. x [M * share, K]."""
    x = widen(x)
    M, K = x.shape[0] // share, x.shape[1]
    h, size = np.zeros((M, K)), np.zeros((M, K))
    if residual is not None:
        h += widen(residual)
        size += np.abs(widen(residual))
    for j in range(share):
        row = x[j::share]
        if weights is not None:
            w = np.asarray(weights, dtype=np.float64)[:, j:j + 1]
            row = np.where(w == 0, 0.0, w * np.where(w == 0, 0.0, row))
        h += row
        size += np.abs(row)
    return h, size


def norm(h, gamma, eps):
    """y of rows h [M, K]; rows of zeros with eps 0 give 0."""
    ms = (h * h).mean(1, keepdims=True) + float(np.float32(eps))
    with np.errstate(divide="ignore"):
        r = np.where(ms > 0, 1 / np.sqrt(ms), 0.0)
    return h * r * np.asarray(gamma, dtype=np.float64)


def sigmoid(z):
    """1 / (1 + exp(-z)) without overflow."""
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def gelu_u(g):
    return math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)


def act(gate, up, gelu):
    """f(gate) up in f64."""
    g = widen(gate)
    f = g * sigmoid(2 * gelu_u(g)) if gelu else g * sigmoid(g)
    return f if up is None else f * widen(up)


def act_tolerance(gate, up, gelu, bf16):
    """include/q4.h, q4_act. By its operations, u = 2^-24 the half step of f32: the
    exponent z log2 e is a product with a rounded constant, off by 1.25 u of itself
    (the constant log2 e is off by 2^-26.2) for SiLU and by 4 u for GELU (g^2, the
    constants, the sum, the product), so exp(-z) by |z| times that (z = g, or 2 u);
    the exponential by 2 u, 1 + e by u, the quotient by 2 u and a little, the product
    with up by u. 2^-20 is 16 u, |g| 2^-23 twice and |u| 2^-20 twice the shares of z."""
    y = np.abs(act(gate, up, gelu))
    g = widen(gate)
    rel = 2.0 ** -20 + (2.0 ** -20 * np.abs(gelu_u(g)) if gelu else 2.0 ** -23 * np.abs(g))
    u = 1.0 if up is None else np.abs(widen(up))
    # In bfloat16 the f32 result is rounded once more, by half a step at most.
    half = 2.0 ** -8 * (y * (1 + rel)) if bf16 else 0.0
    return rel * y + u * 2.0 ** -119 + 2.0 ** -149 + half + (2.0 ** -134 if bf16 else 0.0)


def route(logits, bias, top_k, sigmoid_scores, n_groups, top_groups, group_best, renorm, scale):
    """ids, weights [T, top_k] in f64, offsets [E + 1], order [T top_k]."""
    x = np.asarray(logits, dtype=np.float32).astype(np.float64)
    T, E = x.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float32).astype(np.float64)
    there = x > -np.inf                                  # NaN masks too
    if sigmoid_scores:
        s = np.where(there, sigmoid(np.clip(np.where(there, x, 0.0), -700, 700)), 0.0)
    else:
        top = np.where(there, x, -np.inf).max(1, keepdims=True)
        d = np.where(there, x, 0.0) - np.where(np.isinf(top), 0.0, top)
        s = np.where(there, np.exp(np.maximum(d, -700)), 0.0)
        total = s.sum(1, keepdims=True)
        s = np.divide(s, total, out=np.zeros_like(s), where=total > 0)
    open_ = there & (b > -np.inf)[None, :]
    key = np.where(open_, s + np.where(b > -np.inf, b, 0.0), -np.inf)
    ids, weights = np.zeros((T, top_k), dtype=np.int64), np.zeros((T, top_k))
    size = E // n_groups
    for t in range(T):
        kept = np.arange(E)
        if top_groups < n_groups:
            best = np.sort(key[t].reshape(n_groups, size), axis=1)[:, ::-1][:, :group_best].sum(1)
            groups = np.argsort(-best, kind="stable")[:top_groups]
            kept = np.sort(np.concatenate([np.arange(g * size, (g + 1) * size) for g in groups]))
        ids[t] = kept[np.argsort(-key[t][kept], kind="stable")[:top_k]]
        w = np.where(open_[t, ids[t]], s[t, ids[t]], 0.0)
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
        weights[t] = w * float(np.float32(scale))
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    return ids, weights, offsets, order
