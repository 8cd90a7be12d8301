"""The plain forms of plain_experts.py against hand values and torch's own
conversions (CPU)."""
import numpy as np
import pytest
import torch

import plain_experts as pl


def test_e4m3_values_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).float().numpy()
    got = pl.e4m3_decode(codes)
    assert np.array_equal(np.isnan(ref), np.isnan(got))
    fine = ~np.isnan(ref)
    assert np.array_equal(ref[fine], got[fine].astype(np.float32))
    assert got[0x7E] == 448 and got[0x01] == 2.0 ** -9 and got[0x08] == 2.0 ** -6


def test_encode_matches_torch_and_rounds_ties_to_even():
    rng = np.random.default_rng(1)
    grid = pl.TABLE[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    x = np.concatenate([grid, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9),
                        rng.uniform(-448, 448, 20000), rng.normal(0, 0.01, 20000)]).astype(np.float32)
    x = np.concatenate([x, -x])
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(pl.e4m3_encode(x), ref)
    assert pl.e4m3_encode(np.float32([1.0625]))[0] == 0x38     # between 1 and 1.125: to even
    assert pl.e4m3_encode(np.float32([1.1875]))[0] == 0x3A


def test_quantize_hand_block():
    x = np.zeros((2, 160), dtype=np.float32)
    x[0, 0], x[0, 1], x[0, 130] = 896.0, -3.0, 448.0
    q, s = pl.quantize(x, 1)
    assert s.tolist() == [[2.0, 1.0], [0.0, 0.0]]
    assert q[0, 0] == 0x7E and pl.e4m3_decode(q[0, 1]) == -1.5 and q[0, 130] == 0x7E
    q, s = pl.quantize(x, 128)
    assert s.tolist() == [[2.0, 1.0]]


def test_bf16_bits_match_torch():
    rng = np.random.default_rng(2)
    x = np.concatenate([rng.normal(size=1000), [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]]).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(pl.bf16_bits(x), ref)


def test_product_one_hot():
    a, a_s = pl.quantize(np.eye(3, 160, 129, dtype=np.float32), 1)
    w = np.random.default_rng(3).normal(size=(5, 160)).astype(np.float32)
    wq, w_s = pl.quantize(w, 128)
    y, P = pl.product(a, a_s, wq, w_s)
    assert np.allclose(y, pl.dequant(wq, w_s, 128)[:, 129:132].T, rtol=1e-7, atol=0)
    assert np.allclose(P, np.abs(y))


@pytest.mark.parametrize("renorm", [True, False])
def test_route_hand(renorm):
    x = [[0.0, 2.0, 2.0, 1.0], [5.0, -np.inf, 5.0, 5.0]]
    ids, w, off, order = pl.route(x, 2, renorm)
    assert ids.tolist() == [[1, 2], [0, 2]]
    assert off.tolist() == [0, 1, 2, 4, 4] and order.tolist() == [2, 0, 1, 3]
    assert np.allclose(w.sum(1), 1.0) == renorm
    assert np.allclose(w[1], 0.5 if renorm else 1 / 3)
    ids, w, off, order = pl.route([[-np.inf] * 3], 2, renorm)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]
