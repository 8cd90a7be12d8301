"""Rows named twice in the grouped products' lists where K is cut into segments,
on the GPU against the plain 64-bit forms (plain_experts.py)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import oracle  # noqa: E402
import plain_experts as pl  # noqa: E402
from test_gpu_experts import FORMS, activations, run_grouped, weights  # noqa: E402


def is_one_of(fmt, y, r, groups, av, wv, K):
    """Element by element: row r is the product with one of the groups' weights."""
    ok = np.zeros(y.shape[1], dtype=bool)
    for e in groups:
        ref, P = wv[e] @ av[r], np.abs(wv[e]) @ np.abs(av[r])
        ok |= np.abs(y[r] - ref) <= (pl.product_tolerance(ref, P, K) if fmt == "f8" else oracle.tolerance(P))
    return ok.all()


@pytest.mark.parametrize("fmt,act", FORMS)
@pytest.mark.parametrize("K", [14464, 14592])
def test_rows_named_twice_at_long_k(fmt, act, K):
    # Three K segments. Group 0 names rows 5 and 6 twice; groups 0 and 2 overlap,
    # and group 3 names row 2 of group 0 again.
    G, M, N = 4, 150, 270
    off = [0, 40, 30, 140, M]                     # [0, 40), none, [40, 140) less its clamp, [140, 150)
    order = np.arange(M)
    order[[20, 21, 145]] = [5, 6, 2]
    off[3] = 140
    a, av = activations(act, M, K, 21)
    w, wv = weights(fmt, G, N, K, 300)
    named = [set() for _ in range(M)]
    lo = 0
    for e in range(G):
        first = min(max(off[e], 0), M)
        for p in range(first, max(min(off[e + 1], M), first)):
            named[order[p]].add(e)
    y = run_grouped(fmt, act, a, w, off, order, 1, G, M, N, K)
    assert any(len(n) > 1 for n in named) and any(not n for n in named)
    for r in range(M):
        if named[r]:
            assert is_one_of(fmt, y, r, named[r], av, wv, K), r
        else:
            assert (y[r] == 7.0).all(), r


@pytest.mark.parametrize("fmt,act", FORMS)
def test_every_group_claims_every_row_at_long_k(fmt, act):
    G, M, N, K = 8, 150, 300, 14592
    a, av = activations(act, M, K, 22)
    w, wv = weights(fmt, G, N, K, 330)
    y = run_grouped(fmt, act, a, w, [0, M] * (G // 2) + [0], None, 1, G, M, N, K)
    ok = y == 7.0
    for e in range(0, G, 2):
        ref, P = av @ wv[e].T, np.abs(av) @ np.abs(wv[e]).T
        ok |= np.abs(y - ref) <= (pl.product_tolerance(ref, P, K) if fmt == "f8" else oracle.tolerance(P))
    assert ok.all() and (y != 7.0).any()
