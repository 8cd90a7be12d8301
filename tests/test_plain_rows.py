"""Pins of the plain forms in plain_rows.py: hand-worked values, and torch's own
64-bit operations where it has them."""
import math

import numpy as np
import torch

import plain_rows as plain


def test_norm_by_hand():
    x = np.array([[1, 2], [3, 4], [5, 6], [7, 8]], dtype=np.float32)
    w = np.array([[0.5, 0.25], [1, 0]], dtype=np.float32)
    res = np.array([[10, 0], [0, 1]], dtype=np.float32)
    h, size = plain.norm_sum(x, w, 2, res)
    assert np.array_equal(h, [[11.25, 2], [5, 7]]) and np.array_equal(size, h)
    h, _ = plain.norm_sum(x, None, 2, None)
    assert np.array_equal(h, [[4, 6], [12, 14]])
    h, _ = plain.norm_sum(np.array([[1, np.nan], [2, 3]], dtype=np.float32), np.array([[0, 1]], dtype=np.float32), 2, None)
    assert np.array_equal(h, [[2, 3]])
    y = plain.norm(np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)], [0, 0]], rtol=1e-15)
    y = plain.norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.5)
    assert np.allclose(y, [[3 / math.sqrt(13), 8 / math.sqrt(13)]], rtol=1e-15)


def test_act_against_torch():
    g, u = np.linspace(-30, 30, 401).astype(np.float32)[:, None], np.full((401, 1), 1.5, dtype=np.float32)
    t = torch.from_numpy(g).double()
    assert np.allclose(plain.act(g, u, False), (torch.nn.functional.silu(t) * 1.5).numpy(), rtol=1e-14, atol=0)
    # torch's tanh form loses the last bits of 1 + tanh where that is small.
    want = (torch.nn.functional.gelu(t, approximate="tanh") * 1.5).numpy()
    assert np.allclose(plain.act(g, u, True), want, rtol=1e-12, atol=1e-14)
    assert np.array_equal(plain.act(g, None, True) * 1.5, plain.act(g, u, True))
    assert np.array_equal(plain.widen(np.array([0x3F80, 0xC000], dtype=np.uint16)), [1.0, -2.0])


def test_route_by_hand():
    x = np.log(np.array([[1, 3, 1, 1 / 3, 9, 1]], dtype=np.float64)).astype(np.float32)   # scores 1/2 3/4 1/2 1/4 9/10 1/2
    ids, w, off, order = plain.route(x, None, 3, True, 1, 1, 1, False, 1.0)
    assert ids.tolist() == [[4, 1, 0]] and np.allclose(w, [[0.9, 0.75, 0.5]], rtol=1e-6)
    assert off.tolist() == [0, 1, 2, 2, 2, 3, 3] and order.tolist() == [2, 1, 0]
    ids, w, _, _ = plain.route(x, np.array([0, 0, 0, 1, 0, 0], dtype=np.float32), 2, True, 1, 1, 1, True, 2.0)
    assert ids.tolist() == [[3, 4]] and np.allclose(w, [[0.5 / 1.15, 1.8 / 1.15]], rtol=1e-6)
    # Groups of two: their best 3/4, 1/2, 9/10; their best two 5/4, 3/4, 7/5.
    ids, _, _, _ = plain.route(x, None, 2, True, 3, 1, 1, True, 1.0)
    assert ids.tolist() == [[4, 5]]
    ids, _, _, _ = plain.route(x, None, 4, True, 3, 2, 2, True, 1.0)
    assert ids.tolist() == [[4, 1, 0, 5]]
    # Softmax: shares of 1 + 3 + 1 + 1/3 + 9 + 1.
    ids, w, _, _ = plain.route(x, None, 2, False, 1, 1, 1, False, 1.0)
    assert ids.tolist() == [[4, 1]] and np.allclose(w, [[9 / (46 / 3), 3 / (46 / 3)]], rtol=1e-6)
    # Masks: by the logit, by NaN and by the bias; masked ones come last with weight 0.
    x = np.array([[0, -np.inf, np.nan, 1], [-np.inf] * 4], dtype=np.float32)
    ids, w, _, _ = plain.route(x, np.array([-np.inf, 0, 0, 0], dtype=np.float32), 3, True, 1, 1, 1, True, 1.0)
    assert ids.tolist() == [[3, 0, 1], [0, 1, 2]] and w.tolist() == [[1, 0, 0], [0, 0, 0]]
