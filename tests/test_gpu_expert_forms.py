"""Every kernel form of the E4M3 products and of the products grouped by expert
(expert_cases.py, which test_expert_forms.py holds to the library's rules):
exact sums, scales of every block, what follows a short block, wrong and
overlapping lists, streams and captured graphs."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import expert_cases as cases  # noqa: E402
import oracle  # noqa: E402
import plain_experts as pl  # noqa: E402
from block_quantized_weight_dequant_amd import binding as q4  # noqa: E402
from block_quantized_weight_dequant_amd import workloads as wl  # noqa: E402
from gpu_helpers import DEV, Guarded, to_dev  # noqa: E402
from test_gpu_experts import activations, check_grouped, run_grouped, split, weights  # noqa: E402
from test_gpu_f8 import check, quantized, run_product, values  # noqa: E402

F8 = [pytest.param(*s, id="%s-%dx%dx%d" % ((f,) + s)) for f, l in cases.F8.items() for s in l]
F8_GROUPED = [pytest.param(*s, id="%s-%d" % (f, s[1])) for f, l in cases.F8_GROUPED.items() for s in l]
BLOCK_QUANTIZED = [("q4", "f32"), ("q4", "bf16"), ("q8", "f32"), ("q8", "bf16")]


def small_codes(rng, *shape):
    return pl.e4m3_encode(rng.integers(-4, 5, shape).astype(np.float32))


def rounded(ref):
    return pl.bf16_value(pl.bf16_bits(ref.astype(np.float32))).reshape(ref.shape)


# ---------------------------------------------------------------------------
# E4M3 products

@pytest.mark.parametrize("M,N,K", F8)
def test_f8_sums_of_small_integers_are_exact(M, N, K):
    # Codes of 0, +-1 .. +-4, a power of two a row: whole numbers below 2^15 of
    # it, so only y's rounding is left.
    rng = np.random.default_rng(M + K)
    a, w = small_codes(rng, M, K), small_codes(rng, N, K)
    a_s = np.repeat(np.exp2(rng.integers(-3, 4, (M, 1))), pl.blocks(K), 1).astype(np.float32)
    w_s = np.full((pl.blocks(N), pl.blocks(K)), 0.25, dtype=np.float32)
    ref, _ = pl.product(a, a_s, w, w_s)
    assert np.array_equal(run_product(q4.f8_gemm, a, a_s, w, w_s, M, N, K), rounded(ref))


@pytest.mark.parametrize("M,N,K", F8)
def test_f8_every_block_has_its_own_scales(M, N, K):
    # A one-hot row picks one block of one row: its two scales, and a code.
    rng = np.random.default_rng(M + N)
    a = np.zeros((M, K), dtype=np.uint8)
    a[np.arange(M), rng.integers(0, K, M)] = 0x38     # 1.0
    a_s = np.exp2(rng.integers(-8, 8, (M, pl.blocks(K)))).astype(np.float32)
    w, _ = quantized(7, N, K, 128)
    w_s = np.exp2(rng.integers(-8, 8, (pl.blocks(N), pl.blocks(K)))).astype(np.float32)
    ref, _ = pl.product(a, a_s, w, w_s)
    assert np.array_equal(run_product(q4.f8_gemm, a, a_s, w, w_s, M, N, K), ref)   # four bits: nothing is rounded


@pytest.mark.parametrize("M,N,K", F8)
def test_f8_values_past_a_short_block_do_not_count(M, N, K):
    # What follows a row in memory is the next row, here NaN codes; K % 128 != 0.
    rng = np.random.default_rng(M)
    a, w = small_codes(rng, M, K), small_codes(rng, N, K)
    a[1::2], w[1::2] = 0x7F, 0x7F
    a_s, w_s = np.ones((M, pl.blocks(K)), np.float32), np.ones((pl.blocks(N), pl.blocks(K)), np.float32)
    y = run_product(q4.f8_gemm, a, a_s, w, w_s, M, N, K)
    A, W = pl.e4m3_decode(a[::2]), pl.e4m3_decode(w[::2])
    assert np.array_equal(y[::2, ::2], rounded(A @ W.T))
    assert np.isnan(y[1::2]).all() and np.isnan(y[:, 1::2]).all()


@pytest.mark.parametrize("M,N,K", F8)
def test_f8_normal_values(M, N, K):
    a, a_s = quantized(M, M, K, 1)
    w, w_s = quantized(N + 1, N, K, 128)
    ref, P = pl.product(a, a_s, w, w_s)
    check(run_product(q4.f8_gemm, a, a_s, w, w_s, M, N, K), ref, P, K, "gemm")


@pytest.mark.parametrize("M,N,K", F8)
def test_f8_side_stream_and_graph(M, N, K):
    w, w_s = (to_dev(t) for t in quantized(11, N, K, 128))
    x = to_dev(values(12, M, K))
    qa, qs = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(M, pl.blocks(K), device=DEV)
    y = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.f8_quantize(x, qa, qs, M, K)
        q4.f8_gemm(qa, qs, w, w_s, y, M, N, K)
    s = torch.cuda.Stream()
    for seed in (13, 14, 15):
        x.copy_(to_dev(values(seed, M, K)))
        graph.replay()
        torch.cuda.synchronize()
        ea, es, ey = torch.empty_like(qa), torch.empty_like(qs), torch.zeros_like(y)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            q4.f8_quantize(x, ea, es, M, K)
            q4.f8_gemm(ea, es, w, w_s, ey, M, N, K)
        torch.cuda.synchronize()
        assert torch.equal(y, ey)


# ---------------------------------------------------------------------------
# E4M3 grouped by expert

def f8_small(counts, N, K, share, extra, seed):
    G = len(counts)
    off, n = split(counts)
    M, rng = n + extra, np.random.default_rng(seed)
    T = -(-M // share)
    a, w = small_codes(rng, T, K), small_codes(rng, G, N, K)
    a_s = np.exp2(rng.integers(-3, 4, (T, 1))).repeat(pl.blocks(K), 1).astype(np.float32)
    w_s = np.exp2(rng.integers(-2, 3, (G, 1, 1))).repeat(pl.blocks(N), 1).repeat(pl.blocks(K), 2).astype(np.float32)
    av = pl.e4m3_decode(a) * a_s[:, :1]
    wv = pl.e4m3_decode(w) * w_s[:, :1, :1]
    return G, M, off, (a, a_s), (w, w_s), av, wv, rng.permutation(M)


def by_group(av, wv, off, order, share, M):
    """y of every position's row, and which rows there are: numpy, whole groups at a time."""
    y, there = np.full((M, wv.shape[1]), 7.0), np.zeros(M, dtype=bool)
    for e in range(len(off) - 1):
        rows = np.arange(off[e], off[e + 1]) if order is None else order[off[e]:off[e + 1]]
        y[rows], there[rows] = av[rows // share] @ wv[e].T, True
    return y, there


@pytest.mark.parametrize("counts,N,K,share,extra", F8_GROUPED)
def test_f8_grouped_sums_of_small_integers_are_exact(counts, N, K, share, extra):
    G, M, off, a, w, av, wv, order = f8_small(counts, N, K, share, extra, N + K)
    for o in (order, None):
        ref, there = by_group(av, wv, off, o, share, M)
        assert there.sum() == M - extra
        y = run_grouped("f8", "f8", a, w, off, o, share, G, M, N, K)
        assert np.array_equal(y, rounded(ref))       # 7.0 in the rows of no group


@pytest.mark.parametrize("counts,N,K,share,extra", F8_GROUPED)
def test_f8_grouped_wrong_lists_stay_in_bounds(counts, N, K, share, extra):
    # Groups that overlap, a bound past M, rows outside [0, M), rows named twice.
    G, M, off, a, w, av, wv, order = f8_small(counts, N, K, share, extra, N)
    order[[0, M // 2]], order[[1, M - 1]] = [-1, M], order[[2, 2]]
    off = off.copy()
    off[1], off[-1] = M // 2, 2 ** 31 - 1
    y = run_grouped("f8", "f8", a, w, off, order, share, G, M, N, K)
    ok = y == 7.0
    for e in range(G):
        lo = min(max(int(off[e]), 0), M)
        rows = order[lo:max(min(int(off[e + 1]), M), lo)]
        rows = rows[(rows >= 0) & (rows < M)]
        ok[rows] |= y[rows] == rounded(av[rows // share] @ wv[e].T)
    assert ok.all() and (y != 7.0).any()


# ---------------------------------------------------------------------------
# Q4_0 and Q8_0 grouped by expert

def reference(av, wv, off, order, share, M):
    y, there = by_group(av, wv, off, order, share, M)
    P, _ = by_group(np.abs(av), np.abs(wv), off, order, share, M)
    return y, P, there


@pytest.mark.parametrize("fmt,act", BLOCK_QUANTIZED)
@pytest.mark.parametrize("counts,N,K,share,extra", cases.TILES)
def test_grouped_tiles(fmt, act, counts, N, K, share, extra):
    G = len(counts)
    off, n = split(counts)
    M = n + extra
    order = np.random.default_rng(M + N).permutation(M)
    a, av = activations(act, -(-M // share), K, 11)
    w, wv = weights(fmt, G, N, K, 1000)
    for o in (order, None):
        ref, P, there = reference(av, wv, off, o, share, M)
        assert there.sum() == n
        check_grouped(fmt, run_grouped(fmt, act, a, w, off, o, share, G, M, N, K), ref, P, there, K, o is None)


@pytest.mark.parametrize("fmt,act,form", [(f, act, form) for f in ("q4", "q8") for act in ("f32", "bf16") for form in cases.FEW[f]])
def test_grouped_few_rows(fmt, act, form):
    for counts, N, K, share, extra in cases.FEW[fmt][form]:
        G = len(counts)
        off, n = split(counts)
        M = n + extra
        order = np.random.default_rng(M + N).permutation(M)
        a, av = activations(act, -(-M // share), K, 12)
        w, wv = weights(fmt, G, N, K, 1100)
        ref, P, there = reference(av, wv, off, order, share, M)
        check_grouped(fmt, run_grouped(fmt, act, a, w, off, order, share, G, M, N, K), ref, P, there, K, form)


def one_of_its_groups(y, off, order, av, wv, share, M):
    ok = y == 7.0
    for e in range(len(off) - 1):
        lo = min(max(off[e], 0), M)
        hi = max(min(off[e + 1], M), lo)
        rows = np.arange(lo, hi) if order is None else order[lo:hi]
        rows = rows[(rows >= 0) & (rows < M)]
        A = av[rows // share]
        ok[rows] |= np.abs(y[rows] - A @ wv[e].T) <= oracle.tolerance(np.abs(A) @ np.abs(wv[e]).T)
    return ok.all()


@pytest.mark.parametrize("fmt,act", BLOCK_QUANTIZED)
@pytest.mark.parametrize("K", [384, 512])
def test_grouped_tiles_of_wrong_lists_stay_in_bounds(fmt, act, K):
    G, M, N = 4, 600, 3300
    a, av = activations(act, M, K, 14)
    w, wv = weights(fmt, G, N, K, 55)
    order = np.random.default_rng(K).permutation(M)
    order[[2, 400]], order[[20, 21]] = [-5, 2 ** 30], order[5]
    off = [-7, 300, 150, 590, 2 ** 31 - 1]           # [0, 300), none, [150, 590), [590, 600)
    y = run_grouped(fmt, act, a, w, off, order, 1, G, M, N, K)
    assert one_of_its_groups(y, off, order, av, wv, 1, M)
    named = order[(order >= 0) & (order < M)]
    assert (y[named] != 7.0).any(1).all() and (y[np.setdiff1d(np.arange(M), named)] == 7.0).all()
    # Every other group claims every row: more row tiles than the workspace holds.
    off = [0, M, 0, M, 0]
    y = run_grouped(fmt, act, a, w, off, None, 1, G, M, N, K)
    assert one_of_its_groups(y, off, None, av, wv, 1, M) and (y != 7.0).any()


@pytest.mark.parametrize("fmt,act", BLOCK_QUANTIZED)
@pytest.mark.parametrize("T,E,k,N,K", cases.TILE_LAYERS)
def test_grouped_tiles_on_streams_and_captured(fmt, act, T, E, k, N, K):
    # Router into the grouped product, captured with a workspace of its own;
    # replayed with new inputs between eager calls on side streams.
    S = T * k
    w, wv = weights(fmt, E, N, K, 500)
    dw = to_dev(w)
    name = fmt + "_gemm_grouped" + ("_bf16" if act == "bf16" else "")
    f, need = getattr(q4, name), getattr(q4, name + "_workspace_bytes")(E, S, N, K)
    x = torch.zeros(T, K, dtype=torch.bfloat16 if act == "bf16" else torch.float32, device=DEV)
    logits = torch.zeros(T, E, device=DEV)
    e = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device=DEV)
    i = torch.int32
    ids, wt, off, order, rws = e(S, dtype=i), e(S), e(E + 1, dtype=i), e(S, dtype=i), e(
        max(1, q4.q4_route_workspace_bytes(T, E, k)), dtype=torch.uint8)
    ws, y = torch.empty(need, dtype=torch.uint8, device=DEV), e(S, N)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4_route(logits, ids, wt, off, order, T, E, k, workspace=rws)
        f(x, dw, off, order, y, E, S, N, K, share=k, workspace=ws)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for seed in (4, 5, 6):
        x.copy_(to_dev(wl.activations_f32(seed, T, K)).to(x.dtype))
        lg = wl.activations_f32(seed + 10, T, E)
        logits.copy_(to_dev(lg))
        graph.replay()
        torch.cuda.synchronize()
        outs = []
        for n in range(6):
            s, out = streams[n % 3], torch.zeros_like(y)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                f(x, dw, off, order, out, E, S, N, K, share=k, workspace=torch.full_like(ws, 0xFF))   # NaN patterns
            outs.append(out)
        torch.cuda.synchronize()
        assert all(torch.equal(out, y) for out in outs)
        _, _, ho, hr = pl.route(lg, k, True)
        ref, P, _ = reference(x.double().cpu().numpy(), wv, ho, hr, k, S)
        assert (np.abs(y.cpu().numpy() - ref) <= oracle.tolerance(P)).all()


@pytest.mark.parametrize("fmt,act", BLOCK_QUANTIZED)
def test_grouped_tiles_match_one_product_per_group(fmt, act):
    G, N, K = 3, 3300, 640
    counts = [200, 0, 390]
    off, M = split(counts)
    a, av = activations(act, M, K, 16)
    w, wv = weights(fmt, G, N, K, 57)
    y = run_grouped(fmt, act, a, w, off, None, 1, G, M, N, K)
    f = getattr(q4, fmt + ("_gemm_bf16" if act == "bf16" else "_gemm_ws"))
    for e in (0, 2):
        lo, hi = int(off[e]), int(off[e + 1])
        one = torch.empty(hi - lo, N, device=DEV)
        f(to_dev(a[lo:hi]), to_dev(w[e]), one, hi - lo, N, K)
        torch.cuda.synchronize()
        # The same operands, the same order of sums.
        assert np.array_equal(one.cpu().numpy(), y[lo:hi].astype(np.float32))
