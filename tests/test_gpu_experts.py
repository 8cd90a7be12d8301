"""The router and the grouped products on the GPU against the plain 64-bit forms
(plain_experts.py) and the oracle's block decode."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import oracle  # noqa: E402
import plain_experts as pl  # noqa: E402
from block_quantized_weight_dequant_amd import binding as q4  # noqa: E402
from block_quantized_weight_dequant_amd import workloads as wl  # noqa: E402
from gpu_helpers import DEV, Guarded, to_dev  # noqa: E402


# ---------------------------------------------------------------------------
# Router

def run_route(x, T, E, k, renorm, **kw):
    S = T * k
    ids, off, order = (Guarded(n, torch.int32) for n in (S, E + 1, S))
    w = Guarded(S, torch.float32)
    q4.q4_route(to_dev(x), ids.view, w.view, off.view, order.view, T, E, k, renorm, **kw)
    torch.cuda.synchronize()
    assert all(g.guards_intact() for g in (ids, off, order, w))
    return ids.host().reshape(T, k), w.host().reshape(T, k), off.host(), order.host()


def check_route(x, got, k, renorm):
    T, E = x.shape
    ids, w, off, order = pl.route(x, k, renorm)
    assert np.array_equal(got[0], ids)
    assert np.array_equal(got[2], off) and np.array_equal(got[3], order)
    # exp in f32 (at most 2 steps off), its argument rounded once (|l - max| <
    # 104 where exp is not 0, 2^-24 relative: 104 2^-24), a sum and a division.
    assert (np.abs(got[1] - w) <= (E + 120) * 2.0 ** -24 * w + 2.0 ** -126).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 7, 7), (31, 64, 6), (64, 8, 2), (65, 8, 2), (100, 65, 32),
                                   (257, 128, 8), (300, 200, 4), (130, 256, 32), (77, 1024, 5), (9000, 40, 6), (66000, 8, 1)])
def test_route(T, E, k, renorm):
    rng = np.random.default_rng(T + E)
    x = rng.normal(size=(T, E)).astype(np.float32)
    if T % 2:       # equal logits: bfloat16 values, few of them
        x = np.round(x * 2) / 2
    check_route(x, run_route(x, T, E, k, renorm), k, renorm)


@pytest.mark.parametrize("T", [5, 150])
def test_route_masks_and_extremes(T):
    E, k = 24, 4
    rng = np.random.default_rng(3)
    x = rng.normal(size=(T, E)).astype(np.float32) * 50
    x[rng.random((T, E)) < 0.6] = -np.inf
    x[0] = -np.inf                       # every expert masked
    x[1] = 0.0
    x[1, 3::2] = -0.0                    # equal: the lowest expert, not the +0
    x[2], x[2, 5], x[2, 9] = -3.4e38, 3.4e38, -np.inf
    x[3], x[3, 20] = -np.inf, -7.0       # one expert left
    x[4] = 1e-45
    for renorm in (True, False):
        check_route(x, run_route(x, T, E, k, renorm), k, renorm)


@pytest.mark.parametrize("T", [3, 200])
def test_route_of_nan_is_still_a_grouping(T):
    E, k = 16, 5
    x = np.full((T, E), np.nan, dtype=np.float32)
    x[1, :8] = -np.nan
    x[2] = np.inf
    ids, _, off, order = run_route(x, T, E, k, True)
    assert all(len(set(r)) == k and 0 <= min(r) and max(r) < E for r in ids.tolist())
    assert np.array_equal(order, np.argsort(ids.reshape(-1), kind="stable"))
    assert off[0] == 0 and off[-1] == T * k


def test_route_every_token_to_one_expert():
    x = np.zeros((1000, 32), dtype=np.float32)
    x[:, 17] = 1
    got = run_route(x, 1000, 32, 1, True)
    check_route(x, got, 1, True)
    assert got[2][17] == 0 and got[2][18] == 1000


# ---------------------------------------------------------------------------
# Grouped products

def weights(fmt, G, N, K, seed):
    """(device argument(s), decoded f64 [G, N, K])."""
    if fmt == "f8":
        q, s = zip(*(pl.quantize(wl.weights_f32(seed + e, N, K), 128) for e in range(G)))
        return (np.stack(q), np.stack(s)), np.stack([pl.dequant(a, b, 128) for a, b in zip(q, s)])
    blobs = [getattr(oracle, fmt + "_0_quantize")(wl.weights_f32(seed + e, N, K)) for e in range(G)]
    return np.stack(blobs), np.stack([getattr(oracle, fmt + "_0_dequant")(b).reshape(N, K) for b in blobs]).astype(np.float64)


def activations(act, R, K, seed):
    """(device argument(s), f64 values [R, K])."""
    x = wl.activations_f32(seed, R, K)
    if act == "f8":
        q, s = pl.quantize(x, 1)
        return (q, s), pl.dequant(q, s, 1)
    if act == "bf16":
        bits = pl.bf16_bits(x)
        return bits.view(np.int16), pl.bf16_value(bits).astype(np.float64)
    return x, x.astype(np.float64)


FORMS = [("q4", "f32"), ("q4", "bf16"), ("q8", "f32"), ("q8", "bf16"), ("f8", "f8")]


def run_grouped(fmt, act, a, w, offsets, order, share, G, M, N, K, y=None, **kw):
    off = to_dev(np.asarray(offsets, dtype=np.int32))
    order = None if order is None else to_dev(np.asarray(order, dtype=np.int32))
    y = y or Guarded(M * N, torch.bfloat16 if fmt == "f8" else torch.float32, fill=7.0)
    if fmt == "f8":
        q4.f8_gemm_grouped(to_dev(a[0]), to_dev(a[1]), to_dev(w[0]), to_dev(w[1]), off, order, y.view, G, M, N, K, share=share, **kw)
    else:
        f = getattr(q4, fmt + "_gemm_grouped" + ("_bf16" if act == "bf16" else ""))
        f(to_dev(a), to_dev(w), off, order, y.view, G, M, N, K, share=share, **kw)
    torch.cuda.synchronize()
    assert y.guards_intact()
    return y.view.float().cpu().numpy().reshape(M, N).astype(np.float64)


def check_grouped(fmt, y, ref, P, there, K, what):
    assert (y[~there] == 7.0).all(), what          # rows in no group are left as they were
    tol = pl.product_tolerance(ref, P, K) if fmt == "f8" else oracle.tolerance(P)
    err = np.abs(y - ref)[there]
    assert np.isfinite(y).all() and (err <= tol[there]).all(), (what, float((err / tol[there]).max()))


def split(counts, M=None):
    off = np.concatenate([[0], np.cumsum(counts)])
    return off, int(off[-1]) if M is None else M


CASES = [
    # counts of the groups, N, K, share, extra rows in no group
    ([1], 1, 64, 1, 0),
    ([1, 0, 1, 0], 100, 256, 2, 0),
    ([0, 0, 5, 0, 17], 130, 512, 1, 3),
    ([3, 16, 17, 1], 48, 1024, 3, 0),
    ([33, 0, 2, 15], 200, 768, 1, 1),
    ([40, 31, 64, 0, 1], 33, 4352, 2, 0),
    ([2, 3], 65, 448, 1, 0),
    ([130, 1, 0, 260], 140, 320, 1, 2),
    ([200, 129], 257, 1088, 2, 0),
    ([30, 20, 25], 40, 512, 1, 0),
    ([1] * 70, 20, 256, 1, 0),
    ([33, 0, 2, 15], 70, 704, 1, 2),
    ([0] * 20 + [90] + [1] * 10, 130, 1088, 2, 1),
    ([7, 30], 300, 64, 1, 0),
    ([0] * 100 + [9] + [0] * 30 + [4], 40, 512, 1, 0),
]


@pytest.mark.parametrize("fmt,act", FORMS)
@pytest.mark.parametrize("counts,N,K,share,extra", CASES)
def test_grouped(fmt, act, counts, N, K, share, extra):
    G = len(counts)
    off, n = split(counts)
    M = n + extra
    rng = np.random.default_rng(M + N)
    order = rng.permutation(M)
    a, av = activations(act, -(-M // share), K, 11)
    w, wv = weights(fmt, G, N, K, 1000)
    ref, P, there = pl.grouped(av, wv, off, order, share, M)
    assert there.sum() == n
    y = run_grouped(fmt, act, a, w, off, order, share, G, M, N, K)
    check_grouped(fmt, y, ref, P, there, K, "order")
    ref, P, there = pl.grouped(av, wv, off, None, share, M)
    check_grouped(fmt, run_grouped(fmt, act, a, w, off, None, share, G, M, N, K), ref, P, there, K, "sorted")


@pytest.mark.parametrize("fmt,act", FORMS)
def test_grouped_wide_form(fmt, act):
    # Enough weight rows for the widest few-row workgroups, one and two subtiles.
    G, N, K = 4, 16400, 256
    w, wv = weights(fmt, G, N, K, 77)
    for counts in ([5, 0, 16, 2], [20, 30, 1, 17], [64, 3, 40, 0]):
        off, M = split(counts)
        a, av = activations(act, M, K, 12)
        order = np.random.default_rng(1).permutation(M)
        ref, P, there = pl.grouped(av, wv, off, order, 1, M)
        check_grouped(fmt, run_grouped(fmt, act, a, w, off, order, 1, G, M, N, K), ref, P, there, K, counts)


@pytest.mark.parametrize("counts,N,K", [([150, 3, 247], 4104, 416), ([500, 3, 197], 4100, 288), ([500, 20], 8192, 1056),
                                        ([3000, 900], 8192, 160), ([60, 50, 64, 0, 40], 14336, 672)])
def test_grouped_f8_tile_forms(counts, N, K):
    # Enough rows and columns for each form of larger tiles; the reference in
    # f64 on the card.
    G, (off, M) = len(counts), split(counts)
    g = torch.Generator(device=DEV).manual_seed(5)
    x, v = torch.randn(M, K, generator=g, device=DEV), torch.randn(G * N, K, generator=g, device=DEV)
    a, a_s, A = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(M, pl.blocks(K), device=DEV), torch.empty(M, K, device=DEV)
    q4.f8_quantize(x, a, a_s, M, K)
    q4.f8_dequant(a, a_s, A, M, K)
    w = torch.empty(G, N, K, dtype=torch.uint8, device=DEV)
    w_s = torch.empty(G, pl.blocks(N), pl.blocks(K), device=DEV)
    W = torch.empty(G, N, K, device=DEV)
    for e in range(G):
        s = torch.empty(pl.blocks(N), pl.blocks(K), device=DEV)     # w_s[e] need not be 16-byte aligned
        q4.f8_quantize(v[e * N:(e + 1) * N], w[e], s, N, K, 128)
        q4.f8_dequant(w[e], s, W[e], N, K, 128)
        w_s[e] = s
    order = torch.randperm(M, generator=g, device=DEV)
    ref, P = torch.empty(M, N, dtype=torch.float64, device=DEV), torch.empty(M, N, dtype=torch.float64, device=DEV)
    for e in range(G):
        rows = order[int(off[e]):int(off[e + 1])]
        B = W[e].double().t().contiguous()
        ref[rows], P[rows] = A[rows].double() @ B, A[rows].double().abs() @ B.abs()
    y = Guarded(M * N, torch.bfloat16, fill=7.0)
    q4.f8_gemm_grouped(a, a_s, w, w_s, to_dev(np.asarray(off, dtype=np.int32)), order.int(), y.view, G, M, N, K)
    torch.cuda.synchronize()
    assert y.guards_intact()
    tol = 1.01 * pl.product_tolerance(ref.cpu().numpy(), P.cpu().numpy(), K)     # A and W are rounded to f32
    err = (y.view.double().reshape(M, N) - ref).abs().cpu().numpy()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("fmt,act", [("q4", "f32"), ("q8", "bf16"), ("f8", "f8")])
@pytest.mark.parametrize("M,K", [(6, 28928), (300, 28928), (40, 14336), (40, 14592)])
def test_grouped_long_rows(fmt, act, M, K):
    # K = 14336 is the few-row form's longest; two and more K segments of the tiles.
    N, G = 40, 2
    off, _ = split([M - 2, 2])
    a, av = activations(act, M, K, 13)
    w, wv = weights(fmt, G, N, K, 99)
    ref, P, there = pl.grouped(av, wv, off, None, 1, M)
    check_grouped(fmt, run_grouped(fmt, act, a, w, off, None, 1, G, M, N, K), ref, P, there, K, "long")


@pytest.mark.parametrize("fmt,act", FORMS)
@pytest.mark.parametrize("K", [256, 320])
def test_grouped_wrong_lists_stay_in_bounds(fmt, act, K):
    # Bounds that fall or pass M, rows outside [0, M), a row named twice: the
    # rows that are named rightly get their values.
    G, M, N = 3, 20, 48
    a, av = activations(act, M, K, 14)
    w, wv = weights(fmt, G, N, K, 55)
    order = np.arange(M)
    order[[2, 9]] = [-5, 2 ** 30]
    offsets = [-7, 12, 4, 2 ** 31 - 1]          # groups [0, 12), none, [4, 20): positions 4..11 are in two
    y = run_grouped(fmt, act, a, w, offsets, order, 1, G, M, N, K)
    tol = lambda ref, P: pl.product_tolerance(ref, P, K) if fmt == "f8" else oracle.tolerance(P)
    for rows, e in (([0, 1, 3], [0]), (range(12, 20), [2]), ([4, 5, 6, 7, 8, 10, 11], [0, 2])):
        for r in rows:
            ok = np.zeros(N, dtype=bool)
            for g in e:
                ref, P = wv[g] @ av[r], np.abs(wv[g]) @ np.abs(av[r])
                ok |= np.abs(y[r] - ref) <= tol(ref, P)
            assert ok.all(), r
    assert (y[[2, 9]] == 7.0).all()


@pytest.mark.parametrize("fmt,act", FORMS)
@pytest.mark.parametrize("K", [256, 320])
def test_grouped_overlapping_groups_stay_in_bounds(fmt, act, K):
    # Bounds that fall again and again: every other group claims every row, far
    # more row tiles than M rows have. Each element is one group's value or
    # was left alone.
    G, M, N = 40, 150, 48
    a, av = activations(act, M, K, 20)
    w, wv = weights(fmt, G, N, K, 61)
    y = run_grouped(fmt, act, a, w, [0, M] * (G // 2) + [0], None, 1, G, M, N, K)
    ok = y == 7.0
    for e in range(0, G, 2):
        ref, P = av @ wv[e].T, np.abs(av) @ np.abs(wv[e]).T
        ok |= np.abs(y - ref) <= (pl.product_tolerance(ref, P, K) if fmt == "f8" else oracle.tolerance(P))
    assert ok.all() and (y != 7.0).any()


@pytest.mark.parametrize("fmt,act", FORMS)
def test_grouped_no_rows_at_all(fmt, act):
    G, M, N, K = 2, 5, 32, 256
    a, _ = activations(act, M, K, 15)
    w, _ = weights(fmt, G, N, K, 56)
    assert (run_grouped(fmt, act, a, w, [0, 0, 0], None, 1, G, M, N, K) == 7.0).all()
    assert (run_grouped(fmt, act, a, w, [5, 5, 5], None, 1, G, M, N, K) == 7.0).all()


@pytest.mark.parametrize("fmt,act", FORMS)
@pytest.mark.parametrize("M", [37, 400])
def test_grouped_matches_one_product_per_group(fmt, act, M):
    # Against the library's own product of each group's rows.
    G, N, K = 3, 160, 512
    counts = [M // 3, 0, M - M // 3]
    off, _ = split(counts)
    a, av = activations(act, M, K, 16)
    w, wv = weights(fmt, G, N, K, 57)
    y = run_grouped(fmt, act, a, w, off, None, 1, G, M, N, K)
    for e in range(G):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        m = int(hi - lo)
        if fmt == "f8":
            one = torch.empty(m, N, dtype=torch.bfloat16, device=DEV)
            q4.f8_gemm(to_dev(a[0][lo:hi]), to_dev(a[1][lo:hi]), to_dev(w[0][e]), to_dev(w[1][e]), one, m, N, K)
        else:
            one = torch.empty(m, N, device=DEV)
            f = getattr(q4, fmt + ("_gemm_bf16" if act == "bf16" else "_gemm_ws"))
            f(to_dev(a[lo:hi]), to_dev(w[e]), one, m, N, K)
        torch.cuda.synchronize()
        d = np.abs(one.float().cpu().numpy().astype(np.float64) - y[lo:hi])
        P = np.abs(av[lo:hi]) @ np.abs(wv[e]).T
        ref = av[lo:hi] @ wv[e].T
        tol = pl.product_tolerance(ref, P, K) if fmt == "f8" else oracle.tolerance(P)
        assert (d <= 2 * tol).all()


# ---------------------------------------------------------------------------
# Together

def expert_layer(x, logits, w1, w1s, w2, w2s, T, E, k, H, D, buf, stream=None):
    """Router, quantize, up products, quantize, down products; buffers of the caller."""
    S = T * k
    q4.q4_route(logits, buf["ids"], buf["weights"], buf["offsets"], buf["order"], T, E, k, workspace=buf["ws"], stream=stream)
    q4.f8_quantize_bf16(x, buf["xq"], buf["xs"], T, D, stream=stream)
    q4.f8_gemm_grouped(buf["xq"], buf["xs"], w1, w1s, buf["offsets"], buf["order"], buf["h"], E, S, H, D, share=k, stream=stream)
    q4.f8_quantize_bf16(buf["h"], buf["hq"], buf["hs"], S, H, stream=stream)
    q4.f8_gemm_grouped(buf["hq"], buf["hs"], w2, w2s, buf["offsets"], buf["order"], buf["y"], E, S, D, H, share=1, stream=stream)


def layer_buffers(T, E, k, H, D):
    S, e = T * k, lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device=DEV)
    i, u, b = torch.int32, torch.uint8, torch.bfloat16
    return dict(ids=e(S, dtype=i), weights=e(S), offsets=e(E + 1, dtype=i), order=e(S, dtype=i),
                ws=e(max(1, q4.q4_route_workspace_bytes(T, E, k)), dtype=u), xq=e(T, D, dtype=u), xs=e(T, pl.blocks(D)),
                h=e(S, H, dtype=b), hq=e(S, H, dtype=u), hs=e(S, pl.blocks(H)), y=e(S, D, dtype=b))


@pytest.mark.parametrize("T,E,k,H,D", [(1, 4, 2, 160, 256), (50, 8, 2, 288, 384), (300, 6, 3, 256, 160)])
def test_expert_layer_eager_and_captured(T, E, k, H, D):
    w1, w1v = weights("f8", E, H, D, 300)
    w2, w2v = weights("f8", E, D, H, 400)
    dw = [to_dev(t) for t in (*w1, *w2)]
    x, logits = torch.zeros(T, D, dtype=torch.bfloat16, device=DEV), torch.zeros(T, E, device=DEV)
    cap, eager = layer_buffers(T, E, k, H, D), layer_buffers(T, E, k, H, D)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        expert_layer(x, logits, *dw, T, E, k, H, D, cap)
    for seed in (1, 2, 3):
        rng = np.random.default_rng(seed)
        bits = pl.bf16_bits(rng.normal(size=(T, D)).astype(np.float32))
        lg = rng.normal(size=(T, E)).astype(np.float32)
        x.copy_(to_dev(bits.view(np.int16)).view(torch.bfloat16))
        logits.copy_(to_dev(lg))
        graph.replay()
        torch.cuda.synchronize()
        expert_layer(x, logits, *dw, T, E, k, H, D, eager)
        torch.cuda.synchronize()
        for name in ("ids", "weights", "offsets", "order", "h", "y"):
            assert torch.equal(cap[name], eager[name]), (seed, name)
        # Each step against its plain form on the step's own inputs.
        ids, w, off, order = pl.route(lg, k, True)
        assert np.array_equal(cap["order"].cpu().numpy(), order)
        q, s = pl.quantize(pl.bf16_value(bits), 1)
        ref, P, there = pl.grouped(pl.dequant(q, s, 1), w1v, off, order, k, T * k)
        h = cap["h"].float().cpu().numpy()
        check_grouped("f8", h.astype(np.float64), ref, P, there, D, "up")
        q, s = pl.quantize(h, 1)
        ref, P, there = pl.grouped(pl.dequant(q, s, 1), w2v, off, order, 1, T * k)
        check_grouped("f8", cap["y"].float().cpu().numpy().astype(np.float64), ref, P, there, H, "down")


@pytest.mark.parametrize("fmt,act", FORMS)
@pytest.mark.parametrize("T,N,K", [(3, 300, 512), (37, 520, 1088), (300, 2048, 512)])
def test_grouped_calls_on_several_streams_at_once(fmt, act, T, N, K):
    # Each call has its own workspace, from the allocator's pool of the stream it
    # runs on; the weights, lists and activations are shared.
    E, k = 6, 2
    S = T * k
    a, _ = activations(act, T, K, 31)
    w, _ = weights(fmt, E, N, K, 700)
    rng = np.random.default_rng(T)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].reshape(-1)
    off = to_dev(np.searchsorted(np.sort(ids), np.arange(E + 1)).astype(np.int32))
    order = to_dev(np.argsort(ids, kind="stable").astype(np.int32))
    if fmt == "f8":
        args = [to_dev(t) for t in (a[0], a[1], w[0], w[1])]
        f, dtype = q4.f8_gemm_grouped, torch.bfloat16
    else:
        args = [to_dev(a), to_dev(w)]
        f, dtype = getattr(q4, fmt + "_gemm_grouped" + ("_bf16" if act == "bf16" else "")), torch.float32
    y = torch.empty(S, N, dtype=dtype, device=DEV)
    f(*args, off, order, y, E, S, N, K, share=k)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(9):
        s, out = streams[i % 3], torch.zeros(S, N, dtype=dtype, device=DEV)
        s.wait_stream(torch.cuda.current_stream())
        if i % 2:
            with torch.cuda.stream(s):
                f(*args, off, order, out, E, S, N, K, share=k)
        else:
            f(*args, off, order, out, E, S, N, K, share=k, stream=s)
        outs.append(out)
    torch.cuda.synchronize()
    assert all(torch.equal(out, y) for out in outs)


@pytest.mark.parametrize("fmt,act", [("q4", "bf16"), ("q8", "f32")])
@pytest.mark.parametrize("T", [3, 200])
def test_routed_block_quantized_products_captured(fmt, act, T):
    # Router into the grouped product of every slot's expert, captured with a
    # workspace of its own, replayed with new inputs between eager calls.
    E, k, N, K = 5, 2, 144, 512
    S = T * k
    w, wv = weights(fmt, E, N, K, 500)
    dw = to_dev(w)
    name = fmt + "_gemm_grouped" + ("_bf16" if act == "bf16" else "")
    f, need = getattr(q4, name), getattr(q4, name + "_workspace_bytes")(E, S, N, K)
    x = torch.zeros(T, K, dtype=torch.bfloat16 if act == "bf16" else torch.float32, device=DEV)
    logits = torch.zeros(T, E, device=DEV)
    buf = layer_buffers(T, E, k, 32, 32)
    ws, y = torch.empty(need, dtype=torch.uint8, device=DEV), torch.zeros(S, N, device=DEV)

    def layer(y, ws):
        q4.q4_route(logits, buf["ids"], buf["weights"], buf["offsets"], buf["order"], T, E, k, workspace=buf["ws"])
        f(x, dw, buf["offsets"], buf["order"], y, E, S, N, K, share=k, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(y, ws)
    for seed in (4, 5, 6):
        xv = wl.activations_f32(seed, T, K)
        lg = wl.activations_f32(seed + 10, T, E)
        x.copy_(to_dev(xv).to(x.dtype))
        logits.copy_(to_dev(lg))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        other = torch.zeros_like(y)
        layer(other, torch.full_like(ws, 0xFF))          # a workspace of NaN patterns
        torch.cuda.synchronize()
        assert torch.equal(got, other)
        ids, _, off, order = pl.route(lg, k, True)
        ref, P, _ = pl.grouped(x.double().cpu().numpy(), wv, off, order, k, S)
        assert (np.abs(got.cpu().numpy() - ref) <= oracle.tolerance(P)).all()


def test_side_streams_with_their_own_workspaces():
    G, M, N, K = 3, 45, 96, 512
    off, _ = split([20, 5, 20])
    a, av = activations("f32", M, K, 18)
    w, wv = weights("q4", G, N, K, 58)
    ref, P, there = pl.grouped(av, wv, off, None, 1, M)
    da, dw, do = to_dev(a), to_dev(w), to_dev(off.astype(np.int32))
    streams = [torch.cuda.Stream() for _ in range(3)]
    ys = [torch.zeros(M, N, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, y in zip(streams, ys):
            q4.q4_gemm_grouped(da, dw, do, None, y, G, M, N, K, stream=s)
    torch.cuda.synchronize()
    for y in ys:
        assert torch.equal(y, ys[0])
        assert (np.abs(y.cpu().numpy() - ref) <= oracle.tolerance(P)).all()
