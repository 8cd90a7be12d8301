"""Edges of the E4M3 quantizer on the GPU: signed zeros under scales of every
size and quotients a step past 448, against the plain form (plain_experts.py), bit for bit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import plain_experts as pl  # noqa: E402
from block_quantized_weight_dequant_amd import binding as q4  # noqa: E402
from gpu_helpers import Guarded, f32_bits, to_dev  # noqa: E402


def check_codes(x, block_rows, act):
    M, K = x.shape
    ref_q, ref_s = pl.quantize(x, block_rows)
    q, s = Guarded(M * K, torch.uint8), Guarded(ref_s.size, torch.float32)
    if act == "bf16":
        bits = pl.bf16_bits(x)
        assert np.array_equal(pl.bf16_value(bits).reshape(M, K), x)
        q4.f8_quantize_bf16(to_dev(bits.view(np.int16)), q.view, s.view, M, K, block_rows)
    else:
        q4.f8_quantize(to_dev(x), q.view, s.view, M, K, block_rows)
    torch.cuda.synchronize()
    assert np.array_equal(f32_bits(s.host()), f32_bits(ref_s).reshape(-1))
    assert np.array_equal(q.host().reshape(M, K), ref_q)
    assert q.guards_intact() and s.guards_intact()
    return ref_q


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** 100])
def test_quantize_keeps_the_sign_of_zero(block_rows, act, scale):
    # -0 / s is -0, code 0x80, whatever the scale; so is a negative quotient
    # that rounds to zero.
    rng = np.random.default_rng(9)
    x = rng.choice(np.float32([1.0, -0.5, 0.0, -0.0, 2.0 ** -20, -2.0 ** -20]), (9, 160)) * np.float32(scale)
    x[:, 0] = scale
    q = check_codes(x.astype(np.float32), block_rows, act)
    assert (q == 0x80).any() and (q == 0).any()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_of_maxima_a_step_past_448(block_rows):
    # max / s in f32, s = max / 448 in f32, can be 448 + 2^-15 for ordinary
    # scales: it is still the code of 448.
    v = np.random.default_rng(10).uniform(1, 8, 4096).astype(np.float32)
    v = np.concatenate([np.float32([1.921268, 3.9120002]), v])
    past = v / (v / np.float32(448)) > 448
    assert past[:2].all() and past.sum() > 100
    v = v[past][:101]
    x = np.zeros((101 * block_rows, 128), dtype=np.float32)
    x[::block_rows, 3], x[::block_rows, 77] = v, -v
    q = check_codes(x, block_rows, "f32")
    assert (q[::block_rows, 3] == 0x7E).all() and (q[::block_rows, 77] == 0xFE).all()


@pytest.mark.parametrize("M,N,K", [(5, 100, 160), (40, 4096, 160), (140, 3900, 288), (520, 4096, 160), (975, 8200, 160)])
def test_product_of_scales_below_the_normal_range(M, N, K):
    # a_s w_s of 2^-145 to 2^-135: formed in f32, a multiple of 2^-149 (off by
    # 2^-150 at most), so each block is off by 2^-150 of its codes' sum more.
    # Each of the blocks' additions and y's rounding to bfloat16 add half a step
    # below the normal range: 2^-150 a block, 2^-134.
    rng = np.random.default_rng(M)
    a = pl.e4m3_encode(rng.normal(size=(M, K)).astype(np.float32) * 100)
    w = pl.e4m3_encode(rng.normal(size=(N, K)).astype(np.float32) * 100)
    a_s = np.exp2(rng.uniform(-72, -68, (M, pl.blocks(K)))).astype(np.float32)
    w_s = np.exp2(rng.uniform(-73, -67, (pl.blocks(N), pl.blocks(K)))).astype(np.float32)
    ref, P = pl.product(a, a_s, w, w_s)
    C = np.abs(pl.e4m3_decode(a)) @ np.abs(pl.e4m3_decode(w)).T
    y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    q4.f8_gemm(to_dev(a), to_dev(a_s), to_dev(w), to_dev(w_s), y, M, N, K)
    torch.cuda.synchronize()
    tol = pl.product_tolerance(ref, P, K) + 2.0 ** -150 * (1.01 * C + 2 * pl.blocks(K)) + 2.0 ** -134
    got = y.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol).all() and (got != 0).mean() > 0.9
