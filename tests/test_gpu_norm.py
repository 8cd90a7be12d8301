"""GPU tests of the norms (q4_norm, q8_norm, f8_norm and their bfloat16 forms)
against plain_rows.py in 64 bits.

Tolerances, from include/q4.h. h: half a step of f32 (2^-24) of the exact sum,
and 2^-50 of its terms' sizes for the f64 sums (at most 34 terms of 2^-53). y,
given the h that the call wrote in f32: three roundings of f32 (rstd and two
products, (1 + 2^-24)^3 < 1 + 3.01 2^-24), the f64 mean's and the reciprocal root's
2^-40 at most beside them; where sum is not in f32, h's own rounding counts twice
more (each element's, and rstd's through the mean): 5.02 2^-24. In bfloat16 half a
step, 2^-8, more. 8-bit forms: the bytes that the quantizers make of the f32 y."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import plain_rows as plain  # noqa: E402
from block_quantized_weight_dequant_amd import binding as q4  # noqa: E402
from gpu_helpers import DEV, Guarded, to_dev  # noqa: E402
from plain_experts import bf16_bits  # noqa: E402

U = 2.0 ** -24
EPS = 1e-5


def make(M, K, share, bf16, residual, weighted, seed):
    g = np.random.default_rng(seed)
    rows = np.exp(g.normal(0, 1, (M * share, 1)))
    x = (g.normal(0, 1, (M * share, K)) * rows).astype(np.float32)
    res = (3 * g.normal(0, 1, (M, K))).astype(np.float32) if residual else None
    w = g.uniform(0, 1, (M, share)).astype(np.float32) if weighted else None
    gamma = (1 + 0.2 * g.normal(0, 1, K)).astype(np.float32)
    if bf16:
        x, res = bf16_bits(x), None if res is None else bf16_bits(res)
    return x, res, w, gamma


def dev_of(a):
    if a is None:
        return None
    return to_dev(a.view(np.int16)).view(torch.bfloat16) if a.dtype == np.uint16 else to_dev(a)


def dtype_of(bf16):
    return torch.bfloat16 if bf16 else torch.float32


def host(t):
    """Values in f64."""
    return t.float().cpu().numpy().astype(np.float64)


def check_norm(M, K, share, bf16, residual, weighted, seed, eps=EPS, data=None):
    x, res, w, gamma = data or make(M, K, share, bf16, residual, weighted, seed)
    tail = "_bf16" if bf16 else ""
    what = "M %d K %d share %d %s" % (M, K, share, tail)
    xd, rd, wd, gd = dev_of(x), dev_of(res), dev_of(w), dev_of(gamma)
    kw = dict(residual=rd, weights=wd, share=share)
    norm = getattr(q4, "q4_norm" + tail)
    y32, y16, sm = Guarded(M * K, torch.float32), Guarded(M * K, torch.bfloat16), Guarded(M * K, dtype_of(bf16))
    norm(xd, gd, y32.view, M, K, eps, sum=sm.view, **kw)
    norm(xd, gd, y16.view, M, K, eps, **kw)
    # The 8-bit forms, with and without the sum and the dense result.
    nb = M * (K // 32) * 34
    q8, d8, s8 = Guarded(nb, torch.uint8), Guarded(M * K, dtype_of(bf16)), Guarded(M * K, dtype_of(bf16))
    getattr(q4, "q8_norm" + tail)(xd, gd, q8.view, M, K, eps, y=d8.view, sum=s8.view, **kw)
    ns = M * -(-K // 128)
    f8, fs, df = Guarded(M * K, torch.uint8), Guarded(ns, torch.float32), Guarded(M * K, dtype_of(bf16))
    getattr(q4, "f8_norm" + tail)(xd, gd, f8.view, fs.view, M, K, eps, y=df.view, **kw)
    torch.cuda.synchronize()
    for b in (y32, y16, sm, q8, d8, s8, f8, fs, df):
        assert b.guards_intact(), what

    h, size = plain.norm_sum(x, w, share, res)
    got = host(sm.view).reshape(M, K)
    step = 2.0 ** -8 if bf16 else 0.0
    assert (np.abs(got - h) <= (U + step * (1 + U)) * np.abs(h) + 2.0 ** -50 * size + 2.0 ** -134).all(), what
    y = host(y32.view).reshape(M, K)
    if not bf16:
        ref, rel = plain.norm(got, gamma, eps), 3.01 * U + 2.0 ** -40
        assert (np.abs(y - ref) <= rel * np.abs(ref) + 2.0 ** -126).all(), what
    ref = plain.norm(h, gamma, eps)
    # h's rounding is against the sizes of its terms where they cancel.
    rms = np.sqrt((h * h).mean(1, keepdims=True) + eps)
    loose = 5.02 * U * np.abs(ref) + 2.0 ** -49 * size / np.where(rms > 0, rms, 1) * np.abs(gamma)
    assert (np.abs(y - ref) <= loose + 2.0 ** -126).all(), what
    # Roundings of the same f32 y.
    assert torch.equal(y16.view, y32.view.to(torch.bfloat16)), what
    for d in (d8, df):
        assert torch.equal(d.view, y32.view.to(dtype_of(bf16))), what
    assert torch.equal(s8.view, sm.view), what
    want, ws = torch.empty(nb, dtype=torch.uint8, device=DEV), torch.empty(ns, device=DEV)
    q4.q8_quantize(y32.view.contiguous(), want)
    assert torch.equal(q8.view, want), what
    want = torch.empty(M * K, dtype=torch.uint8, device=DEV)
    q4.f8_quantize(y32.view.contiguous(), want, ws, M, K, 1)
    assert torch.equal(f8.view, want) and torch.equal(fs.view, ws), what


# Four, two and one row a wavefront, 2, 4, 8 and 16 wavefronts a row, several
# pieces a lane; short last blocks of 32 and 128; the widest row.
WIDTHS = [32, 64, 96, 128, 160, 192, 256, 288, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 8192, 8224, 14336, 16416, 32768]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("K", WIDTHS)
def test_widths(K, bf16):
    check_norm(3, K, 1, bf16, True, False, K)
    check_norm(5, K, 2, bf16, True, True, K + 1)
    if K <= 512:
        check_norm(1 + 16 * 5, K, 1, bf16, False, False, K + 2)
        check_norm(2 + 16 * 5, K, 3, bf16, True, True, K + 3)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,K,share,residual,weighted", [
    (1, 4096, 1, True, False), (1, 4096, 8, True, True), (1, 256, 1, False, False), (6, 96, 3, False, True),
    (257, 512, 1, True, False), (1001, 160, 1, True, False), (130, 1056, 32, True, True), (7, 2048, 5, True, False),
    (64, 4096, 1, False, True), (513, 256, 2, False, False), (2050, 2048, 1, True, False),
    (1024, 2336, 1, True, False), (1030, 4128, 1, True, False)])
def test_rows_and_shares(M, K, share, residual, weighted, bf16):
    check_norm(M, K, share, bf16, residual, weighted, 31 * M + K)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("waves", [3, 5, 7, 9, 10, 11, 12, 13, 17, 20, 21, 24, 25])
def test_every_number_of_wavefronts(waves, bf16):
    # A row that ends near the last wavefront's end, and the narrowest.
    lanes = 512 if bf16 else 256
    for K in (waves * lanes - 32, (waves - 1) * lanes + 32):
        check_norm(3, K, 1, bf16, True, False, K)
        check_norm(2, K, 3, bf16, True, True, K + 1)


@pytest.mark.parametrize("bf16", [False, True])
def test_many_rows_of_nine_wavefronts(bf16):
    check_norm(1025, (512 if bf16 else 256) * 9 - 32, 1, bf16, True, False, 77)


@pytest.mark.parametrize("bf16", [False, True])
def test_scales_of_the_data(bf16):
    # Rows of sizes from 2^-60 to 2^60, whose squares leave f32; rows of zeros.
    g = np.random.default_rng(5)
    M, K = 41, 416
    x = (g.normal(0, 1, (M, K)) * np.exp2(np.arange(M)[:, None] * 3.0 - 60)).astype(np.float32)
    x[7] = 0
    gamma = (1 + 0.1 * g.normal(0, 1, K)).astype(np.float32)
    gamma[3] = 0
    for eps in (0.0, 1e-30, 1e-6):
        check_norm(M, K, 1, bf16, False, False, 0, eps=eps, data=(bf16_bits(x) if bf16 else x, None, None, gamma))
    # Below 2^-125, where 1 / rms is past f32, down to the smallest f32.
    x = np.ldexp(g.normal(0, 1, (25, 96)), -125 - np.arange(25)[:, None]).astype(np.float32)
    x[24] = 0
    x[24, 5] = 2.0 ** -133 if bf16 else 2.0 ** -149
    check_norm(25, 96, 1, bf16, False, False, 0, eps=0.0, data=(bf16_bits(x) if bf16 else x, None, None, gamma[:96]))
    big = np.full((2, 64), 1.5e38, dtype=np.float32)
    check_norm(2, 64, 1, bf16, False, False, 0, data=(bf16_bits(big) if bf16 else big, None, None, gamma[:64]))


@pytest.mark.parametrize("bf16", [False, True])
def test_sums_that_cancel(bf16):
    # The experts' rows nearly cancel the residual: f64 sums keep what is left.
    M, K, share = 9, 672, 2
    x, res, w, gamma = make(M, K, share, bf16, True, True, 11)
    terms, _ = plain.norm_sum(x, w, share, None)
    res = -terms.astype(np.float32)
    check_norm(M, K, share, bf16, True, True, 0, data=(x, bf16_bits(res) if bf16 else res, w, gamma))


@pytest.mark.parametrize("bf16", [False, True])
def test_weight_zero_leaves_its_row_out(bf16):
    # Rows of slots in no group hold anything, NaN too.
    M, K, share = 6, 288, 3
    x, res, w, gamma = make(M, K, share, bf16, True, True, 21)
    w[0, 1] = w[2, 0] = w[4, 2] = 0
    w[3] = 0
    w[5, 0] = -0.0
    bad = x.reshape(M, share, K).copy()
    for m, j in [(0, 1), (2, 0), (4, 2), (3, 0), (3, 1), (3, 2), (5, 0)]:
        bad[m, j] = 0x7FC0 if bf16 else np.nan
        bad[m, j, ::7] = 0xFF80 if bf16 else -np.inf
    check_norm(M, K, share, bf16, True, True, 0, data=(bad.reshape(M * share, K), res, w, gamma))
    one = make(4, 96, 1, bf16, True, True, 22)      # one slot a token
    one[2][1, 0] = 0
    one[0][1] = 0x7FC0 if bf16 else np.nan
    check_norm(4, 96, 1, bf16, True, True, 0, data=one)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("K,share", [(64, 9), (1024, 7), (2528, 5), (4096, 3), (5120, 11), (8192, 6), (11616, 13), (32768, 2)])
def test_weight_zero_at_every_width(K, share, bf16):
    M = 2 * share + 1
    x, res, w, gamma = make(M, K, share, bf16, True, True, K)
    for m in range(M):                               # each slot alone, then all but it; the last row: none left
        w[m, m % share if m < share else np.arange(share) != m % share] = 0
    w[-1] = -0.0
    rows = x.reshape(M, share, K)
    rows[w == 0] = 0x7FC0 if bf16 else np.nan
    check_norm(M, K, share, bf16, True, True, 0, data=(x, res, w, gamma))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("share", [1, 4])
def test_sum_in_place(share, bf16):
    M, K = 33, 4128
    x, res, w, gamma = make(M, K, share, bf16, True, share > 1, 3)
    xd, rd, wd, gd = dev_of(x), dev_of(res), dev_of(w), dev_of(gamma)
    apart, y0, y1 = torch.empty_like(rd), torch.empty(M, K, device=DEV), torch.empty(M, K, device=DEV)
    norm = q4.q4_norm_bf16 if bf16 else q4.q4_norm
    norm(xd, gd, y0, M, K, EPS, residual=rd, sum=apart, weights=wd, share=share)
    norm(xd, gd, y1, M, K, EPS, residual=rd, sum=rd, weights=wd, share=share)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(apart, rd)


def test_offsets_past_32_bits():
    # 2^32 elements and more of x and y; the rows near the end, and one before.
    K = 32768
    M = 2 ** 32 // K + 3
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    y = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x.fill_(1.0)
    g = torch.Generator(device=DEV).manual_seed(8)
    tail = torch.randn(4, K, generator=g, device=DEV).to(torch.bfloat16)
    x[-4:] = tail
    gamma = torch.ones(K, device=DEV)
    q4.q4_norm_bf16(x, gamma, y, M, K, EPS)
    torch.cuda.synchronize()
    ref = plain.norm(host(tail), np.ones(K), EPS)
    assert (np.abs(host(y[-4:]) - ref) <= (5.02 * U + 2.0 ** -8 * (1 + 6 * U)) * np.abs(ref) + 2.0 ** -126).all()
    assert bool((y[: M - 4] == 1.0).all())


def test_streams_and_repeats():
    M, K, share = 300, 4096, 2
    x, res, w, gamma = (dev_of(v) for v in make(M, K, share, True, True, True, 40))
    outs = [[torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(M, K // 128, device=DEV),
             torch.empty(M, K, dtype=torch.bfloat16, device=DEV)] for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (q, s, sm), st in zip(outs, [None] + streams):
            q4.f8_norm_bf16(x, gamma, q, s, M, K, EPS, residual=res, sum=sm, weights=w, share=share, stream=st)
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_binding_refuses():
    M, K = 4, 64
    x, gamma, y = torch.zeros(M, K, device=DEV), torch.ones(K, device=DEV), torch.zeros(M, K, device=DEV)
    for args, kw in [((x.cpu(), gamma, y), {}), ((x[:, :32], gamma, y), {}), ((x.t(), gamma, y), {}), ((x.double(), gamma, y), {}),
                     ((x, gamma[:32], y), {}), ((x, gamma, y[:2]), {}), ((x, gamma, y.half()), {}), ((x, gamma, y), dict(share=2)),
                     ((x, gamma, y), dict(residual=x.to(torch.bfloat16))), ((x, gamma, y), dict(weights=torch.ones(M, 2, device=DEV))),
                     ((x, gamma, y), dict(sum=torch.zeros(M, 2 * K, device=DEV)[:, :K]))]:
        with pytest.raises(ValueError):
            q4.q4_norm(*args, M, K, EPS, **kw)
    with pytest.raises(q4.Q4Error) as e:
        q4.q4_norm(x, gamma, x, M, K, EPS)
    assert e.value.status == q4.Q4_ERR_ALIAS
    with pytest.raises(q4.Q4Error) as e:
        q4.q4_norm(x, gamma, y, M, K, -1.0)
    assert e.value.status == q4.Q4_ERR_SHAPE
    with pytest.raises(ValueError):
        q4.q8_norm(x, gamma, torch.zeros(M * 2 * 34 - 1, dtype=torch.uint8, device=DEV), M, K, EPS)
    with pytest.raises(ValueError):
        q4.f8_norm(x, gamma, torch.zeros(M * K, dtype=torch.uint8, device=DEV), torch.zeros(3, device=DEV), M, K, EPS)
    q4.q4_norm(torch.zeros(0, K, device=DEV), gamma, torch.zeros(0, K, device=DEV), 0, K, EPS)   # empty
    torch.cuda.synchronize()
    assert not y.any()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("K", [96, 1056, 4096])
def test_largest_rows(K, bf16):
    # Up to the largest f32, where 1 / rms is below 2^-126: no bits are lost to that. The
    # row in between, and its smallest elements, keep theirs too.
    M = 48
    g = np.random.default_rng(K)
    x = (g.uniform(0.3, 1, (M, K)) * g.choice([-1, 1], (M, K)) * np.exp2(g.uniform(124, 127.95, (M, 1)))).astype(np.float32)
    x[5] = np.float32(3.38e38)
    x[6, ::3] = np.float32(2.0 ** -120)
    x[7] = g.normal(0, 1, K).astype(np.float32)
    gamma = (1 + 0.1 * g.normal(0, 1, K)).astype(np.float32)
    check_norm(M, K, 1, bf16, False, False, 0, data=(bf16_bits(x) if bf16 else x, None, None, gamma))


def test_large_gamma_on_small_elements():
    # h rstd below 2^-126 is off by 2^-150 at most, and gamma times that.
    M, K = 3, 128
    g = np.random.default_rng(3)
    x = g.normal(0, 1, (M, K)).astype(np.float32)
    x[:, ::2] = np.ldexp(g.uniform(0.5, 1, (M, K // 2)), g.integers(-148, -120, (M, K // 2))).astype(np.float32)
    gamma = np.where(np.arange(K) % 2, 1.0, g.uniform(0.5, 1, K) * 2.0 ** 100).astype(np.float32)
    y = torch.empty(M, K, device=DEV)
    q4.q4_norm(to_dev(x), to_dev(gamma), y, M, K, EPS)
    ref = plain.norm(x.astype(np.float64), gamma, float(np.float32(EPS)))
    assert (np.abs(host(y) - ref) <= 2.0 ** -21.6 * np.abs(ref) + 2.0 ** -126 + np.abs(gamma.astype(np.float64)) * 2.0 ** -149).all()


def sampled(M, seed):
    """The rows that are looked at: the first and last ones, and some between."""
    r = np.random.default_rng(seed)
    return np.unique(np.concatenate([np.arange(5), np.arange(M - 5, M), r.integers(0, M, 24)]))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M", [1024, 1025])
@pytest.mark.parametrize("waves", [9, 10, 11, 16])
@pytest.mark.parametrize("share", [1, 2, 3])
def test_many_rows_of_nine_to_sixteen_wavefronts(share, waves, M, bf16):
    # Rows that end near a wavefront's end, and the narrowest, in every form; some
    # weights are 0 over rows of NaN; the sum in place. A sample of the rows against 64
    # bits, all of them against calls of fewer rows (which take other kernels).
    lanes = 512 if bf16 else 256
    dt, tail = dtype_of(bf16), "_bf16" if bf16 else ""
    for K in (waves * lanes - 32, (waves - 1) * lanes + 32):
        g = torch.Generator(device=DEV).manual_seed(M + K + share)
        x = torch.randn(M * share, K, generator=g, device=DEV).to(dt)
        res = (3 * torch.randn(M, K, generator=g, device=DEV)).to(dt)
        gamma = 1 + 0.2 * torch.randn(K, generator=g, device=DEV)
        w = None
        if share > 1:
            w = torch.rand(M, share, generator=g, device=DEV)
            w[torch.rand(M, share, generator=g, device=DEV) < 0.2] = 0
            x[(w == 0).reshape(-1)] = float("nan")
        n, nb, nf = M * K, M * (K // 32) * 34, M * -(-K // 128)
        y32, y16, q8 = Guarded(n, torch.float32), Guarded(n, torch.bfloat16), Guarded(nb, torch.uint8)
        f8, fs, dense = Guarded(n, torch.uint8), Guarded(nf, torch.float32), Guarded(n, dt)
        sm = Guarded(n, dt)
        sm.view.copy_(res.reshape(-1))
        kw = dict(weights=w, share=share)
        getattr(q4, "q4_norm" + tail)(x, gamma, y32.view, M, K, EPS, residual=res, **kw)
        getattr(q4, "q8_norm" + tail)(x, gamma, q8.view, M, K, EPS, residual=res, **kw)
        getattr(q4, "f8_norm" + tail)(x, gamma, f8.view, fs.view, M, K, EPS, residual=res, y=dense.view, **kw)
        getattr(q4, "q4_norm" + tail)(x, gamma, y16.view, M, K, EPS, residual=sm.view, sum=sm.view, **kw)   # in place
        torch.cuda.synchronize()
        what = "M %d K %d share %d %s" % (M, K, share, tail)
        for b in (y32, y16, q8, f8, fs, dense, sm):
            assert b.guards_intact(), what
        at = sampled(M, K)
        pick = lambda t: t.reshape(M, -1)[torch.from_numpy(at).to(DEV)].contiguous()
        xs = pick(x.reshape(M, share * K)).reshape(-1, K)
        bits = (lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)) if bf16 else (lambda t: t.cpu().numpy())
        h, size = plain.norm_sum(bits(xs), None if w is None else pick(w).cpu().numpy(), share, bits(pick(res)))
        step = 2.0 ** -8 if bf16 else 0.0
        got = host(pick(sm.view))
        assert (np.abs(got - h) <= (U + step * (1 + U)) * np.abs(h) + 2.0 ** -50 * size + 2.0 ** -134).all(), what
        ref = plain.norm(h, gamma.cpu().numpy(), EPS)
        rms = np.sqrt((h * h).mean(1, keepdims=True) + EPS)
        loose = 5.02 * U * np.abs(ref) + 2.0 ** -49 * size / rms * np.abs(gamma.cpu().numpy())
        assert (np.abs(host(pick(y32.view)) - ref) <= loose + 2.0 ** -126).all(), what
        # Every row: the same bits as from calls of 300 rows.
        few = torch.empty(n, device=DEV)
        few_sum = torch.empty(M, K, dtype=dt, device=DEV)
        for m0 in range(0, M, 300):
            m1 = min(m0 + 300, M)
            getattr(q4, "q4_norm" + tail)(x[m0 * share:m1 * share], gamma, few[m0 * K:m1 * K], m1 - m0, K, EPS, residual=res[m0:m1],
                                          sum=few_sum[m0:m1], weights=None if w is None else w[m0:m1], share=share)
        assert torch.equal(few_sum.reshape(-1), sm.view), what
        assert torch.equal(few, y32.view), what
        assert torch.equal(y16.view, y32.view.to(torch.bfloat16)) and torch.equal(dense.view, y32.view.to(dt)), what
        want, ws = torch.empty(nb, dtype=torch.uint8, device=DEV), torch.empty(nf, device=DEV)
        q4.q8_quantize(y32.view.contiguous(), want)
        assert torch.equal(q8.view, want), what
        want = torch.empty(n, dtype=torch.uint8, device=DEV)
        q4.f8_quantize(y32.view.contiguous(), want, ws, M, K, 1)
        assert torch.equal(f8.view, want) and torch.equal(fs.view, ws), what


def test_rows_past_a_launch():
    # 2^23 workgroups of 16 rows of 32 columns are 2^27 rows; the rows next to the
    # boundary and the last ones are what calls of their own give, the sum in place.
    M, K = 2 ** 27 + 21, 32
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV).normal_()
    res = torch.ones(M, K, dtype=torch.bfloat16, device=DEV)
    y, gamma = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV), torch.ones(K, device=DEV)
    q4.q4_norm_bf16(x, gamma, y, M, K, EPS, residual=res, sum=res)
    for first, n in ((0, 20), (2 ** 27 - 24, 45), (2 ** 26, 64)):
        want, ws = torch.empty(n, K, dtype=torch.bfloat16, device=DEV), torch.empty(n, K, dtype=torch.bfloat16, device=DEV)
        q4.q4_norm_bf16(x[first:first + n], gamma, want, n, K, EPS, residual=torch.ones_like(ws), sum=ws)
        assert torch.equal(y[first:first + n], want) and torch.equal(res[first:first + n], ws), first
    # No row was added twice, or not at all.
    step = 2 ** 22
    for m in range(0, M, step):
        assert torch.equal(res[m:m + step], (x[m:m + step].float() + 1.0).to(torch.bfloat16)), m
