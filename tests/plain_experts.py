"""Plain 64-bit forms of the E4M3 quantizer, decode and product, of the router
and of the grouped products, for their tests: numpy, written from the
definitions in include/f8.h and include/q4.h. Pinned by test_plain_experts.py."""
import numpy as np

BLOCK = 128


def e4m3_table():
    """The 128 values of the codes 0 .. 127 (0x7F, NaN, last)."""
    v = np.empty(128)
    for c in range(128):
        e, f = c >> 3, c & 7
        v[c] = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
    v[127] = np.nan
    return v


TABLE = e4m3_table()


def e4m3_decode(codes):
    codes = np.asarray(codes, dtype=np.uint8)
    v = TABLE[codes & 127]
    return np.where(codes & 128, -v, v)


def e4m3_encode(x):
    """Nearest code of x in [-448, 448], ties to the even code; x in f32."""
    x = np.asarray(x, dtype=np.float64)
    m, grid = np.abs(x), TABLE[:127]
    hi = np.clip(np.searchsorted(grid, m, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - grid[lo], grid[hi] - m
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def blocks(n):
    return -(-n // BLOCK)


def spread(s, rows, M, K):
    """One scale for each element of [M, K]."""
    return np.repeat(np.repeat(s, rows, 0)[:M], BLOCK, 1)[:, :K]


def quantize(x, block_rows):
    """f32 [M, K] -> codes, scales: the f32 operations of the definition, one by one."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    R = -(-M // block_rows)
    s = np.zeros((R, blocks(K)), dtype=np.float32)
    for r in range(R):
        for b in range(blocks(K)):
            t = x[r * block_rows:(r + 1) * block_rows, b * BLOCK:(b + 1) * BLOCK]
            s[r, b] = np.abs(t).max() / np.float32(448)
    d = spread(s, block_rows, M, K)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        v = np.where(d == 0, np.float32(0), x / d)
    return e4m3_encode(np.clip(v, -448, 448).astype(np.float32)), s


def dequant(q, s, block_rows):
    """f64 values of codes [M, K]."""
    return e4m3_decode(q) * spread(s.astype(np.float64), block_rows, *q.shape)


def product(a, a_s, w, w_s):
    """(a @ w^T, |a| @ |w|^T) in f64."""
    A, W = dequant(a, a_s, 1), dequant(w, w_s, 128)
    return A @ W.T, np.abs(A) @ np.abs(W).T


def product_tolerance(ref, P, K):
    """include/f8.h, f8_gemm: half a step of bfloat16, and the matrix core's
    eight-product sums (7 products cut at 2^-13 of the largest) and f32 adds."""
    return 2.0 ** -8 * np.abs(ref) + 1.01 * (7 * 2.0 ** -13 + (24 + K / 128) * 2.0 ** -23) * P


def bf16_bits(x):
    """Nearest bfloat16 pattern, ties to even, of finite f32 values."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) & 0xFFFF).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32)


def route(logits, top_k, renorm):
    """ids, weights [T, top_k], offsets [E + 1], order [T top_k]: the largest
    logits, the lowest expert among equals, weights in f64."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    ids = np.argsort(-x, axis=1, kind="stable")[:, :top_k]
    with np.errstate(invalid="ignore"):
        p = np.exp(x - x.max(1, keepdims=True))
    p = np.where(np.isnan(p), 0.0, p)          # a row of -inf
    top = np.take_along_axis(p, ids, 1)
    total = top.sum(1, keepdims=True) if renorm else p.sum(1, keepdims=True)
    weights = np.divide(top, total, out=np.zeros_like(top), where=total > 0)
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    return ids, weights, offsets, order


def group_of_positions(offsets, M):
    """Group of each sorted position, -1 outside all of them."""
    g = np.full(M, -1)
    for e in range(len(offsets) - 1):
        g[offsets[e]:offsets[e + 1]] = e
    return g


def grouped(values, weights, offsets, order, share, M):
    """(y, sum |a w|, rows written) of y[r] = values[r // share] @ weights[e]^T."""
    N = weights.shape[1]
    y, P = np.zeros((M, N)), np.zeros((M, N))
    there = np.zeros(M, dtype=bool)
    g = group_of_positions(offsets, M)
    for p in range(M):
        if g[p] < 0:
            continue
        r = p if order is None else order[p]
        a, w = values[r // share], weights[g[p]]
        y[r], P[r], there[r] = w @ a, np.abs(w) @ np.abs(a), True
    return y, P, there
