"""E4M3 quantizer, decode and block-128 product on the GPU against the plain
64-bit forms (plain_experts.py): codes and scales bit for bit, products within
the bound that include/f8.h derives."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import plain_experts as pl  # noqa: E402
from block_quantized_weight_dequant_amd import binding as q4  # noqa: E402
from gpu_helpers import DEV, Guarded, f32_bits, to_dev  # noqa: E402


def values(seed, M, K, kind="normal"):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, K)).astype(np.float32)
    if kind == "wide":          # every block of another size, zeros among them
        x *= np.exp2(rng.integers(-60, 60, (M, pl.blocks(K)))).repeat(128, 1)[:, :K]
        x[rng.random((M, K)) < 0.1] = 0
        x[:, :128][rng.random(M) < 0.3] = 0
    if kind == "edge":          # the largest and the smallest f32, signed zeros, exact ties
        x = rng.choice(np.float32([3.4e38, -3.4e38, 1e-45, -1e-45, 1e-38, 0.0, -0.0, 1.0, 1.0625, -1.1875, 448.0]), (M, K))
        x[:, 128:256] = rng.choice(np.float32([448.0, 1.0625, 1.1875, 0.001953125, 0.0009765625]), x[:, 128:256].shape)
        x[:, 256:384] = rng.choice(np.float32([1e-45, 3e-43, -2e-44, 0]), x[:, 256:384].shape)
    return x


def quantized(seed, M, K, block_rows, kind="normal"):
    return pl.quantize(values(seed, M, K, kind), block_rows)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,kind", [(1, 32, "normal"), (3, 96, "normal"), (5, 160, "wide"), (7, 448, "edge"),
                                      (130, 256, "wide"), (129, 4128, "normal"), (300, 384, "edge"), (2100, 4096, "normal")])
def test_quantize_bit_exact(block_rows, act, M, K, kind):
    x = values(M + K, M, K, kind)
    if act == "bf16":
        bits = pl.bf16_bits(x)
        bits[(bits & 0x7FFF) == 0x7F80] -= 1     # 3.4e38 rounds to infinity
        x, dev, f = pl.bf16_value(bits).reshape(M, K), to_dev(bits.view(np.int16)), q4.f8_quantize_bf16
    else:
        dev, f = to_dev(x), q4.f8_quantize
    ref_q, ref_s = pl.quantize(x, block_rows)
    q, s = Guarded(M * K, torch.uint8), Guarded(ref_s.size, torch.float32)
    f(dev, q.view, s.view, M, K, block_rows)
    torch.cuda.synchronize()
    assert np.array_equal(f32_bits(s.host()), f32_bits(ref_s).reshape(-1))
    assert np.array_equal(q.host().reshape(M, K), ref_q)
    assert q.guards_intact() and s.guards_intact()


@pytest.mark.parametrize("block_rows,M,K", [(1, 1, 32), (1, 9, 160), (128, 131, 288), (128, 1, 96)])
def test_dequant_bit_exact(block_rows, M, K):
    rng = np.random.default_rng(M)
    q = rng.integers(0, 256, (M, K)).astype(np.uint8)
    q[(q & 127) == 127] = 0x7E
    s = np.exp2(rng.uniform(-20, 20, (-(-M // block_rows), pl.blocks(K)))).astype(np.float32)
    out = Guarded(M * K, torch.float32)
    q4.f8_dequant(to_dev(q), to_dev(s), out.view, M, K, block_rows)
    torch.cuda.synchronize()
    ref = (pl.e4m3_decode(q).astype(np.float32) * pl.spread(s, block_rows, M, K)).astype(np.float32)
    assert np.array_equal(f32_bits(out.host()), f32_bits(ref).reshape(-1)) and out.guards_intact()


def run_product(f, a, a_s, w, w_s, M, N, K):
    y = Guarded(M * N, torch.int16)
    f(to_dev(a), to_dev(a_s), to_dev(w), to_dev(w_s), y.view, M, N, K)
    torch.cuda.synchronize()
    assert y.guards_intact()
    return pl.bf16_value(y.host().view(np.uint16)).reshape(M, N).astype(np.float64)


def check(y, ref, P, K, what):
    assert np.isfinite(y).all(), what
    err, tol = np.abs(y - ref), pl.product_tolerance(ref, P, K)
    assert (err <= tol).all(), (what, float((err / tol).max()))


SHAPES = [(1, 1, 32), (1, 16, 128), (1, 100, 160), (1, 257, 1152), (2, 33, 4224), (8, 512, 4096), (9, 30, 96),
          (16, 130, 1024), (17, 64, 288), (31, 129, 2080), (33, 48, 512), (64, 100, 1184), (65, 1, 64), (66, 300, 416),
          (100, 129, 2048), (128, 128, 256), (129, 257, 384), (200, 515, 1120), (513, 140, 4128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["normal", "wide"])
def test_product(M, N, K, kind):
    a, a_s = quantized(M, M, K, 1, kind)
    w, w_s = quantized(N + 1, N, K, 128, kind)
    if kind == "wide":      # keep y inside f32
        a_s, w_s = np.clip(a_s, 0, 1e9).astype(np.float32), np.clip(w_s, 0, 1e9).astype(np.float32)
    ref, P = pl.product(a, a_s, w, w_s)
    check(run_product(q4.f8_gemm, a, a_s, w, w_s, M, N, K), ref, P, K, "gemm")
    if M <= 8:
        check(run_product(q4.f8_gemv, a, a_s, w, w_s, M, N, K), ref, P, K, "gemv")


@pytest.mark.parametrize("M,N,K", [(4, 40, 224), (40, 40, 224), (140, 140, 480)])
def test_product_of_small_integers_is_exact(M, N, K):
    # Codes of 0, +-1 .. +-4 and scales of powers of two: every sum is a whole
    # number of them below 2^13, so only y's rounding is left.
    rng = np.random.default_rng(5)
    a = pl.e4m3_encode(rng.integers(-4, 5, (M, K)).astype(np.float32))
    w = pl.e4m3_encode(rng.integers(-4, 5, (N, K)).astype(np.float32))
    a_s = np.repeat(np.exp2(rng.integers(-3, 4, (M, 1))), pl.blocks(K), 1).astype(np.float32)
    w_s = np.full((pl.blocks(N), pl.blocks(K)), 0.25, dtype=np.float32)
    ref, _ = pl.product(a, a_s, w, w_s)
    y = run_product(q4.f8_gemm, a, a_s, w, w_s, M, N, K)
    assert np.array_equal(y, pl.bf16_value(pl.bf16_bits(ref.astype(np.float32))))


@pytest.mark.parametrize("M", [3, 50, 150])
def test_every_block_has_its_own_scales(M):
    # Scales that differ from block to block and row to row; a one-hot row
    # picks one block.
    N, K = 300, 416
    rng = np.random.default_rng(6)
    a = np.zeros((M, K), dtype=np.uint8)
    hot = rng.integers(0, K, M)
    a[np.arange(M), hot] = 0x38     # 1.0
    a_s = np.exp2(rng.integers(-8, 8, (M, pl.blocks(K)))).astype(np.float32)
    w, _ = quantized(7, N, K, 128)
    w_s = np.exp2(rng.integers(-8, 8, (pl.blocks(N), pl.blocks(K)))).astype(np.float32)
    ref, _ = pl.product(a, a_s, w, w_s)
    y = run_product(q4.f8_gemm, a, a_s, w, w_s, M, N, K)
    assert np.array_equal(y, ref)       # four significant bits: nothing is rounded


def test_values_past_a_short_block_do_not_count():
    # K = 160: the second block of a row is 32 long, and what follows it in
    # memory is the next row, here NaN codes.
    M, N, K = 140, 130, 160
    a, a_s = quantized(8, M, K, 1)
    w, w_s = quantized(9, N, K, 128)
    a[1::2], w[1::2] = 0x7F, 0x7F
    y = run_product(q4.f8_gemm, a, a_s, w, w_s, M, N, K)
    ref, P = pl.product(a[::2], a_s[::2], np.where(w == 0x7F, 0, w), w_s)
    check(y[::2, ::2], ref[:, ::2], P[:, ::2], K, "even rows and columns")
    y = run_product(q4.f8_gemm, a[:60], a_s[:60], w, w_s, 60, N, K)
    check(y[::2, ::2], ref[:30, ::2], P[:30, ::2], K, "few rows")


@pytest.mark.parametrize("M,N,K", [(4096, 4100, 160), (3900, 4096, 1056), (1000, 4104, 288), (300, 14401, 672),
                                   (700, 4100, 1312), (520, 4096, 32), (70, 14400, 1056), (100, 14402, 416), (64, 14336, 1184),
                                   (140, 3900, 416), (130, 2002, 1312), (250, 3008, 160)])
def test_product_large_tiles(M, N, K):
    # Enough rows and columns for each form of tiles (256 x 256, 256 x 128, 128 x
    # 128, 128 x 64, 64 x 64); the reference in f64 on the card.
    g = torch.Generator(device=DEV).manual_seed(3)
    x, v = torch.randn(M, K, generator=g, device=DEV), torch.randn(N, K, generator=g, device=DEV)
    a, a_s = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(M, pl.blocks(K), device=DEV)
    w, w_s = torch.empty(N, K, dtype=torch.uint8, device=DEV), torch.empty(pl.blocks(N), pl.blocks(K), device=DEV)
    q4.f8_quantize(x, a, a_s, M, K)
    q4.f8_quantize(v, w, w_s, N, K, 128)
    A, W = torch.empty(M, K, device=DEV), torch.empty(N, K, device=DEV)
    q4.f8_dequant(a, a_s, A, M, K)
    q4.f8_dequant(w, w_s, W, N, K, 128)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    q4.f8_gemm(a, a_s, w, w_s, y, M, N, K)
    ref, P = A.double() @ W.double().t().contiguous(), A.double().abs() @ W.double().abs().t().contiguous()
    tol = 1.01 * pl.product_tolerance(ref.cpu().numpy(), P.cpu().numpy(), K)     # A and W are rounded to f32
    err = (y.double() - ref).abs().cpu().numpy()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("M", [1, 24, 300])
def test_repeats_side_stream_and_graph(M):
    N, K = 384, 1184
    a, a_s = (to_dev(t) for t in quantized(10, M, K, 1))
    w, w_s = (to_dev(t) for t in quantized(11, N, K, 128))
    y0 = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    q4.f8_gemm(a, a_s, w, w_s, y0, M, N, K)
    x = to_dev(values(12, M, K))
    s = torch.cuda.Stream()
    y1 = torch.zeros_like(y0)
    s.wait_stream(torch.cuda.current_stream())
    q4.f8_gemm(a, a_s, w, w_s, y1, M, N, K, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1)
    # Quantize and multiply, captured; new inputs in the same places.
    qa, qs, y2 = torch.empty_like(a), torch.empty_like(a_s), torch.zeros_like(y0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.f8_quantize(x, qa, qs, M, K)
        q4.f8_gemm(qa, qs, w, w_s, y2, M, N, K)
    for seed in (13, 14, 15):
        x.copy_(to_dev(values(seed, M, K)))
        graph.replay()
        torch.cuda.synchronize()
        got = y2.clone()
        ea, es, ey = torch.empty_like(a), torch.empty_like(a_s), torch.empty_like(y0)
        q4.f8_quantize(x, ea, es, M, K)
        q4.f8_gemm(ea, es, w, w_s, ey, M, N, K)
        torch.cuda.synchronize()
        assert torch.equal(got, ey)
