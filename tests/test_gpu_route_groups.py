"""GPU tests of q4_route_groups against plain_rows.py in 64 bits: choices,
offsets and order exact, weights within one rounding to f32 (2^-24) and 2^-45 for
the f64 scores and their sum."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import plain_rows as plain  # noqa: E402
from block_quantized_weight_dequant_amd import binding as q4  # noqa: E402
from gpu_helpers import DEV, Guarded, to_dev  # noqa: E402


def run(x, bias, k, sigmoid, G=1, top=1, best=1, renorm=True, scale=1.0, stream=None):
    T, E = x.shape
    out = [Guarded(T * k, torch.int32), Guarded(T * k, torch.float32), Guarded(E + 1, torch.int32), Guarded(T * k, torch.int32)]
    q4.q4_route_groups(to_dev(x), None if bias is None else to_dev(bias), *(o.view for o in out), T, E, k,
                       q4.Q4_SCORE_SIGMOID if sigmoid else q4.Q4_SCORE_SOFTMAX, G, top, best, renorm, scale, stream=stream)
    torch.cuda.synchronize()
    assert all(o.guards_intact() for o in out)
    return [o.host() for o in out]


def check(x, bias, k, sigmoid, G=1, top=1, best=1, renorm=True, scale=1.0):
    T, E = x.shape
    what = "T %d E %d k %d sigmoid %s groups %d %d %d renorm %s" % (T, E, k, sigmoid, G, top, best, renorm)
    ids, w, off, order = run(x, bias, k, sigmoid, G, top, best, renorm, scale)
    r_ids, r_w, r_off, r_order = plain.route(x, bias, k, sigmoid, G, top, best, renorm, scale)
    bad = np.argwhere(ids.reshape(T, k) != r_ids)
    assert bad.size == 0, "%s: %d choices differ, first at %s" % (what, len(bad), bad[0])
    assert np.array_equal(off, r_off) and np.array_equal(order, r_order), what
    r_w = r_w.reshape(-1)
    assert (np.abs(w - r_w) <= (2.0 ** -24 + 2.0 ** -45) * np.abs(r_w) + 2.0 ** -149).all(), what


def make(T, E, seed, biased=True):
    g = np.random.default_rng(seed)
    x = (g.normal(0, 1, (T, E)) + 0.5 * g.normal(0, 1, (1, E))).astype(np.float32)
    return x, (0.1 * g.normal(0, 1, E)).astype(np.float32) if biased else None


# One to sixteen experts a lane, group sizes that are and are not powers of two.
SHAPES = [(1, 256, 8, 8, 4, 2), (2, 256, 8, 8, 4, 2), (33, 256, 8, 8, 4, 2), (64, 64, 6, 8, 3, 1), (65, 60, 4, 5, 2, 2),
          (200, 128, 1, 4, 1, 2), (31, 160, 8, 8, 3, 1), (100, 640, 32, 64, 7, 2), (1, 1024, 16, 32, 5, 2), (40, 1000, 10, 10, 9, 2),
          (300, 12, 3, 3, 2, 2), (17, 64, 8, 64, 8, 1), (5, 126, 9, 63, 60, 2), (90, 2, 1, 2, 1, 1), (2100, 256, 8, 8, 4, 2)]


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("T,E,k,G,top,best", SHAPES)
def test_groups(T, E, k, G, top, best, sigmoid):
    x, b = make(T, E, 3 * T + E)
    check(x, b, k, sigmoid, G, top, best, True, 2.5)
    check(x, None, k, sigmoid, G, top, best, False, 1.0)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (64, 8, 2), (77, 65, 7), (130, 256, 32), (9, 257, 8), (200, 1024, 32), (1000, 40, 6)])
def test_no_groups(T, E, k, sigmoid):
    x, b = make(T, E, T + E)
    check(x, b, k, sigmoid, renorm=True, scale=0.5)
    check(x, b, k, sigmoid, renorm=False)
    if E % 2 == 0:
        check(x, b, k, sigmoid, 2, 2, 1)          # all groups kept


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,G,top", [(64, 8, 3), (256, 8, 4), (1000, 10, 4)])
def test_equal_keys(E, G, top, sigmoid):
    # Few distinct logits and biases: the lowest group, then the lowest expert.
    g = np.random.default_rng(E)
    x = (g.integers(-2, 3, (70, E)) * 0.5).astype(np.float32)
    b = (g.integers(0, 2, E) * 0.25).astype(np.float32)
    check(x, b, 8, sigmoid, G, top, 2)
    check(x, None, 8, sigmoid, G, top, 1)
    check(np.zeros((66, E), dtype=np.float32), None, 8, sigmoid, G, top, 2)
    z = np.zeros((3, E), dtype=np.float32)
    z[:, ::3] = -0.0
    check(z, np.where(np.arange(E) % 2, 0.0, -0.0).astype(np.float32), 8, sigmoid, G, top, 2)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_masks(sigmoid):
    T, E, G = 67, 64, 8
    x, b = make(T, E, 77)
    g = np.random.default_rng(1)
    x[g.random((T, E)) < 0.5] = -np.inf
    x[3] = -np.inf                       # nothing left
    x[4, 1:] = -np.inf                   # one expert
    x[5, 8:] = -np.inf                   # one group
    x[6, ::8] = np.nan
    b[[9, 17, 63]] = -np.inf
    b[30] = np.nan
    for G, top, best in [(1, 1, 1), (8, 3, 2), (8, 3, 1), (8, 8, 1)]:
        for renorm in (True, False):
            check(x, b, 6, sigmoid, G, top, best, renorm)
    ids, w, _, _ = run(x, b, 6, sigmoid)
    assert (w.reshape(T, 6)[3] == 0).all() and ids.reshape(T, 6)[3].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("sigmoid", [True, False])
def test_far_logits(sigmoid):
    # Scores down to exp(-700) and saturated ones; beyond, they count as equal.
    g = np.random.default_rng(2)
    x = g.uniform(-690, 5, (130, 128)).astype(np.float32)
    check(x, None, 8, sigmoid, 8, 4, 2)
    x[::2] = g.uniform(-3e4, -1e3, (65, 128)).astype(np.float32)
    check(x, None, 8, sigmoid, 8, 4, 2, renorm=False)
    x = np.full((3, 64), 3.3e38, dtype=np.float32)
    x[1] = -3.3e38
    check(x, None, 4, sigmoid)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,G,top", [(64, 1, 1), (128, 1, 1), (256, 1, 1), (256, 8, 4), (160, 8, 3), (240, 15, 4), (60, 5, 2)])
def test_keys_an_f32_step_apart(E, G, top, biased):
    # Logits some steps of f32 apart, in any order: scores that f32 cannot tell apart,
    # from a few at the edge of the choice to all of them, and groups' sums with them.
    g = np.random.default_rng(E + G)
    T = 96
    x = g.normal(0, 1, (T, E)).astype(np.float32)
    for t in range(T):
        n = [2, 3, 5, 12, 20, E][t % 6]
        at = np.argsort(-x[t], kind="stable")[t % 9:][:n]
        near = np.float32(x[t, at[0]]) + np.arange(len(at)) * np.float32(2.0 ** -23 * (1 + t % 3))
        x[t, at] = g.permutation(near.astype(np.float32))
    b = np.where(g.random(E) < 0.5, np.float32(0.125), np.float32(0.125 + 2.0 ** -24)).astype(np.float32) if biased else None
    for k in (1, 6, 8, 15, 16):
        if k <= top * (E // G):
            check(x, b, k, True, G, top, 2)
            check(x, b, k, False, G, top, 1)


@pytest.mark.parametrize("E,G,top", [(256, 1, 1), (256, 8, 4), (128, 1, 1), (250, 10, 3)])
def test_the_best_are_neighbours(E, G, top):
    # The best sixteen experts side by side, from every start.
    x = np.random.default_rng(3).normal(0, 1, (E - 15, E)).astype(np.float32)
    for t in range(E - 15):
        x[t, t:t + 16] += 6
    for k in (8, 12, 15):
        check(x, None, k, True, G, top, 2)


def test_large_biases_blur_f32():
    # Keys near 10^4 and 10^7, where f32 holds no score.
    x, _ = make(70, 256, 12)
    for size in (1e4, 1e7):
        b = np.full(256, size, dtype=np.float32)
        check(x, b, 8, True, 8, 4, 2)
        b[::3] = -size
        check(x, b, 8, True, 8, 4, 2)
        check(x, b, 8, False, 1, 1, 1)


def test_biases_decide():
    # Large biases of both signs order the experts, the scores weigh them.
    x, _ = make(90, 256, 4)
    b = np.random.default_rng(5).normal(0, 50, 256).astype(np.float32)
    for sigmoid in (True, False):
        check(x, b, 8, sigmoid, 8, 4, 2, True, -1.5)
        check(x, -np.abs(b), 8, sigmoid, 8, 4, 1, False, 0.0)


def test_what_is_not_a_number_stays_a_grouping():
    T, E, k = 100, 256, 8
    x, b = make(T, E, 6)
    x[::3, ::5] = np.nan
    x[::4, 3] = np.inf
    b[7], b[200] = np.nan, np.inf
    ids, _, off, order = run(x, b, k, True, 8, 4, 2)
    ids = ids.reshape(T, k)
    assert ((ids >= 0) & (ids < E)).all() and all(len(set(r)) == k for r in ids.tolist())
    flat = ids.reshape(-1)
    assert np.array_equal(order, np.argsort(flat, kind="stable"))
    assert np.array_equal(off, np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]))


def test_streams_and_repeats():
    x, b = make(3000, 256, 8)
    first = run(x, b, 8, True, 8, 4, 2)
    st = torch.cuda.Stream()
    for s in (None, st, st):
        assert all(np.array_equal(p, q) for p, q in zip(first, run(x, b, 8, True, 8, 4, 2, stream=s)))


def test_binding_refuses():
    T, E, k = 4, 16, 2
    x, i = torch.zeros(T, E, device=DEV), lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)
    ok = [x, None, i(T * k), torch.zeros(T * k, device=DEV), i(E + 1), i(T * k)]
    for at, bad in [(0, x.double()), (0, x[:2]), (0, x.t()), (0, x.cpu()), (1, torch.zeros(E + 1, device=DEV)), (2, i(T * k).long()),
                    (3, i(T * k)), (4, i(E)), (5, i(3))]:
        with pytest.raises(ValueError):
            q4.q4_route_groups(*[bad if j == at else v for j, v in enumerate(ok)], T, E, k)
    with pytest.raises(q4.Q4Error) as e:
        q4.q4_route_groups(*ok, T, E, k, q4.Q4_SCORE_SIGMOID, 3, 1)
    assert e.value.status == q4.Q4_ERR_SHAPE


WIDE = [(512, 1, 1), (512, 8, 4), (320, 8, 3), (272, 16, 4), (257, 1, 1), (510, 15, 5), (320, 10, 2)]   # 17 to 32 experts a lane


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,G,top", WIDE)
def test_wide_rows(E, G, top, sigmoid):
    for T, k in ((1, 1), (33, 8), (66, 15), (300, 6)):
        x, b = make(T, E, T + E)
        check(x, b, k, sigmoid, G, top, 2, True, 2.5)
        check(x, None, k, sigmoid, G, top, 1, False, 1.0)
    test_equal_keys(E, G, top, sigmoid)
    g = np.random.default_rng(E)
    x, b = make(67, E, 77)
    x[g.random((67, E)) < 0.9] = -np.inf
    x[3] = -np.inf
    x[4, 1:] = -np.inf
    x[6, ::8] = np.nan
    b[[9, 17, 63, E - 1]] = -np.inf
    b[30] = np.nan
    check(x, b, 8, sigmoid, G, top, 2)
    check(x, None, 15, sigmoid, G, G, 1)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,G,top", WIDE)
def test_wide_rows_of_near_keys(E, G, top, biased):
    test_keys_an_f32_step_apart(E, G, top, biased)
    if not biased:
        test_the_best_are_neighbours(E, G, top)


@pytest.mark.parametrize("size", [3.0, 50.0, 1e4, 1e7])
def test_wide_rows_with_large_biases(size):
    x, _ = make(70, 512, 12)
    g = np.random.default_rng(5)
    for b in (np.full(512, size, dtype=np.float32), (size * g.normal(0, 1, 512)).astype(np.float32),
              np.where(np.arange(512) % 3, size, -size).astype(np.float32)):
        check(x, b, 8, True, 8, 4, 2)
        check(x, b, 15, True, 1, 1, 1)
        check(x, b, 8, False, 8, 4, 1, False, -1.5)


@pytest.mark.parametrize("B", [0.5, 2.0, 10.0, 100.0, 3000.0])
@pytest.mark.parametrize("E,G,top", [(256, 1, 1), (256, 8, 4), (120, 1, 1), (60, 5, 3), (512, 1, 1), (512, 8, 4)])
def test_near_keys_under_biases_of_both_signs(E, G, top, B):
    # Four experts with the bias B, the others with -B, some of which have scores from a
    # fraction of f32's step at 1 + 2 B to some ten of them apart, at the edge of the
    # choice: the keys' rounding in f32 tells nothing there.
    g = np.random.default_rng(int(10 * B) + E)
    T = 160
    b = np.full(E, -B, dtype=np.float32)
    liked = g.permutation(E)[:4]
    b[liked] = B
    x = (g.normal(0, 1, (T, E)) - 9).astype(np.float32)
    rest = np.setdiff1d(np.arange(E), liked)
    for t in range(T):
        n = int(g.integers(2, 13))
        near = g.permutation(rest)[:n]
        p = g.uniform(0.3, 0.7) + g.permutation(n) * g.uniform(0.02, 3) * (1 + 2 * B) * 2.0 ** -24
        p = np.clip(p, 0.01, 0.99)
        x[t, near] = np.log(p / (1 - p)).astype(np.float32)
    for k in (5, 6, 8, 11, 15):
        if k <= top * (E // G):
            check(x, b, k, True, G, top, 2)
            check(x, b, k, True, G, top, 1)
            check(x, b, k, False, G, top, 2)


def check_many(T, E, k, sigmoid, G=1, top=1, best=1, scale=2.5, seed=0):
    """As check, for many tokens: the definition in torch's 64-bit operations over whole
    arrays (finite logits, no masks)."""
    g = torch.Generator(device=DEV).manual_seed(seed + T + E)
    x = torch.randn(T, E, generator=g, device=DEV)
    b = 0.1 * torch.randn(E, generator=g, device=DEV)
    ids, w, off, order = [Guarded(T * k, torch.int32), Guarded(T * k, torch.float32), Guarded(E + 1, torch.int32), Guarded(T * k, torch.int32)]
    q4.q4_route_groups(x, b, ids.view, w.view, off.view, order.view, T, E, k, q4.Q4_SCORE_SIGMOID if sigmoid else q4.Q4_SCORE_SOFTMAX,
                       G, top, best, True, scale)
    torch.cuda.synchronize()
    assert all(o.guards_intact() for o in (ids, w, off, order))
    s = torch.sigmoid(x.double()) if sigmoid else torch.softmax(x.double(), 1)
    key = s + b.double()
    if top < G:
        sums = torch.sort(key.reshape(T, G, E // G), dim=2, descending=True)[0][:, :, :best].sum(2)
        kept = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        kept.scatter_(1, torch.sort(sums, dim=1, descending=True, stable=True)[1][:, :top], True)
        key = torch.where(kept.repeat_interleave(E // G, 1), key, -torch.inf)
    want = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    what = "T %d E %d k %d" % (T, E, k)
    assert torch.equal(ids.view.reshape(T, k).long(), want), what
    ww = s.gather(1, want)
    ww = scale * ww / ww.sum(1, keepdim=True)
    assert bool(((w.view.reshape(T, k).double() - ww).abs() <= (2.0 ** -24 + 2.0 ** -45) * ww).all()), what
    flat = want.reshape(-1)
    assert torch.equal(order.view.long(), torch.sort(flat, stable=True)[1]), what
    counts = torch.bincount(flat, minlength=E).cpu().numpy()
    assert np.array_equal(off.host(), np.concatenate([[0], np.cumsum(counts)])), what


# Chunks of 33 tokens and more: a second pass of a workgroup's wavefronts, a short one;
# past 64 a third, whose slots start over; a last chunk that ends within a pass.
MANY = [8193, 8200, 8192 + 256 * 5 + 3, 16385, 16700, 25003, 66000]


@pytest.mark.parametrize("T", MANY)
@pytest.mark.parametrize("E,k,G,top,best", [(256, 8, 8, 4, 2), (64, 6, 1, 1, 1), (60, 4, 5, 2, 2), (512, 8, 8, 4, 2), (320, 15, 1, 1, 1),   # rows of lanes
                                            (5, 2, 1, 1, 1),                                                                            # 32-bit counts
                                            (128, 16, 8, 4, 2), (96, 6, 32, 5, 2), (256, 20, 1, 1, 1), (640, 8, 10, 4, 1)])            # a token a wavefront
def test_many_tokens(E, k, G, top, best, T):
    check_many(T, E, k, True, G, top, best)
    if T in (8200, 16700):
        check_many(T, E, k, False, G, top, best)


def test_chunks_whose_counts_may_pass_16_bits():
    # More than 65535 slots a chunk: 32-bit counts of eight experts and more.
    check_many(530000, 32, 32, True)
    check_many(1048577, 16, 16, False)
