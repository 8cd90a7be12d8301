"""The expert layer's products past the threads of one launch (a grid's x
dimension holds fewer than 2^32): many rows of few columns, and many columns
of few rows. Every output must be written and right."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import oracle  # noqa: E402
import plain_experts as pl  # noqa: E402
from block_quantized_weight_dequant_amd import binding as q4  # noqa: E402
from gpu_helpers import DEV, to_dev  # noqa: E402
from test_gpu_experts import activations, weights  # noqa: E402


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def check_shared_rows(y, boundary, per_row, refs, tols):
    """y [M, N]: rows below `boundary` are group 0's, the others group 1's, row
    r that of activation row r // per_row; a block of rows at a time."""
    M = y.shape[0]
    for r0 in range(0, M, per_row):
        t = r0 // per_row
        for e, (lo, hi) in enumerate(((r0, min(r0 + per_row, boundary)), (max(r0, boundary), r0 + per_row))):
            if lo < hi:
                err = (y[lo:hi].double() - refs[e][t]).abs()
                assert bool((err <= tols[e][t]).all()), (t, e)     # also false for NaN


def two_groups(fmt, av, wv, K):
    refs, tols = [], []
    for e in range(2):
        ref, P = av @ wv[e].T, np.abs(av) @ np.abs(wv[e]).T
        refs.append(to_dev(ref))
        tols.append(to_dev(pl.product_tolerance(ref, P, K) if fmt == "f8" else oracle.tolerance(P)))
    return refs, tols


def test_grouped_q4_of_2_29_rows():
    M, N, K, T = 2 ** 29, 8, 64, 64
    a, av = activations("bf16", T, K, 1)
    w, wv = weights("q4", 2, N, K, 2)
    b = M // 3 + 5
    y = torch.full((M, N), float("nan"), device=DEV)
    q4.q4_gemm_grouped_bf16(to_dev(a), to_dev(w), to_dev(np.int32([0, b, M])), None, y, 2, M, N, K, share=M // T)
    torch.cuda.synchronize()
    check_shared_rows(y, b, M // T, *two_groups("q4", av, wv, K))


def test_grouped_f8_of_2_30_rows():
    # One group of more than 2^23 row tiles.
    M, N, K, T = 2 ** 30, 8, 32, 256
    a, av = activations("f8", T, K, 3)
    w, wv = weights("f8", 2, N, K, 4)
    b = M - 1000
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    q4.f8_gemm_grouped(to_dev(a[0]), to_dev(a[1]), to_dev(w[0]), to_dev(w[1]), to_dev(np.int32([0, b, M])), None, y, 2, M, N, K,
                       share=M // T)
    torch.cuda.synchronize()
    check_shared_rows(y, b, M // T, *two_groups("f8", av, wv, K))


def test_f8_product_of_2_29_rows():
    M, N, K = 2 ** 29, 8, 32
    g = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randint(0, 0x7F, (M, K), dtype=torch.uint8, device=DEV, generator=g)
    a_s = torch.rand(M, 1, device=DEV, generator=g)
    w, w_s = pl.quantize(np.random.default_rng(6).normal(size=(N, K)).astype(np.float32), 128)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    q4.f8_gemm(a, a_s, to_dev(w), to_dev(w_s), y, M, N, K)
    torch.cuda.synchronize()
    for r0 in range(0, M, 2 ** 26):
        assert bool(torch.isfinite(y[r0:r0 + 2 ** 26]).all()), r0
    rows = np.unique(np.concatenate([np.arange(200), M - 1 - np.arange(200), np.random.default_rng(7).integers(0, M, 4000)]))
    i = to_dev(rows)
    ref, P = pl.product(a[i].cpu().numpy(), a_s[i].cpu().numpy(), w, w_s)
    err = np.abs(y[i].double().cpu().numpy() - ref)
    assert (err <= pl.product_tolerance(ref, P, K)).all()


def test_grouped_q8_of_2_29_columns():
    M, N, K = 2, 2 ** 29, 64
    g = torch.Generator(device=DEV).manual_seed(8)
    w = torch.randint(0, 256, (N, 2, 34), dtype=torch.uint8, device=DEV, generator=g)
    w[:, :, 0], w[:, :, 1] = 0, 0x24          # d = 2^-6
    a, av = activations("bf16", M, K, 9)
    y = torch.full((M, N), float("nan"), device=DEV)
    q4.q8_gemm_grouped_bf16(to_dev(a), w, to_dev(np.int32([0, M])), None, y, 1, M, N, K)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all())
    cols = np.unique(np.concatenate([np.arange(100), N - 1 - np.arange(100), np.random.default_rng(10).integers(0, N, 4000)]))
    i = to_dev(cols)
    wv = oracle.q8_0_dequant(w[i].reshape(-1).cpu().numpy()).reshape(len(cols), K).astype(np.float64)
    ref, P = av @ wv.T, np.abs(av) @ np.abs(wv).T
    assert (np.abs(y[:, i].cpu().numpy() - ref) <= oracle.tolerance(P)).all()
