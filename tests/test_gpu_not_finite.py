"""GPU tests of NaN and infinities in the rows that the quantizers, the activations
and the norms write in 8 bits: an element that is no number is not stored as one."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from block_quantized_weight_dequant_amd import binding as q4  # noqa: E402
from gpu_helpers import DEV, to_dev  # noqa: E402
from plain_experts import e4m3_decode, spread  # noqa: E402


def dev_of(x, bf16):
    t = to_dev(x)
    return t.to(torch.bfloat16) if bf16 else t


def q8_values(blob, M, K):
    """Values of the Q8_0 blocks [M, K / 32]."""
    b = blob.cpu().numpy().reshape(M, K // 32, 34)
    d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
    with np.errstate(invalid="ignore"):
        return (d * b[..., 2:].view(np.int8)).reshape(M, K)


def f8_values(q, s, M, K, rows=1):
    with np.errstate(invalid="ignore"):
        return e4m3_decode(q.cpu().numpy().reshape(M, K)) * spread(s.cpu().numpy().astype(np.float64).reshape(-(-M // rows), -1), rows, M, K)


def rows_with_faults(M, K):
    """Rows of ordinary and of extreme sizes; (x, where NaN, where infinite)."""
    g = np.random.default_rng(31)
    x = g.normal(0, 1, (M, K)).astype(np.float32)
    x[1] *= np.float32(2.0 ** -100)           # scales outside the range of the reciprocal's quotients
    x[2] *= np.float32(2.0 ** 100)
    x[3] = 0
    nan, inf = np.zeros((M, K), dtype=bool), np.zeros((M, K), dtype=bool)
    for m in range(5):
        nan[m, [5, K - 1]] = True
    nan[5, :128] = True                       # a whole block
    inf[6, 7] = inf[7, K - 3] = True
    return x, nan, inf


def check(got, clean, nan, inf, wide, local):
    """Faults stay visible; blocks of `wide` columns without one are what they are without
    any. local: so are the numbers beside a NaN."""
    M, K = clean.shape
    assert np.isnan(got[nan]).all()
    assert not np.isfinite(got[inf]).any()
    for m in range(M):
        for b in range(0, K, wide):
            at = slice(b, min(b + wide, K))
            ok = ~(nan[m, at] | inf[m, at])
            if ok.all():
                assert np.array_equal(got[m, at], clean[m, at], equal_nan=True), (m, b)
            elif local and not inf[m, at].any():
                assert np.isfinite(got[m, at][ok]).all(), (m, b)


M, K = 9, 416


def test_quantizers():
    x, nan, inf = rows_with_faults(M, K)
    bad = np.where(nan, np.float32(np.nan), np.where(inf, np.float32(-np.inf), x)).astype(np.float32)
    blob, n8 = lambda: torch.empty(M * (K // 32) * 34, dtype=torch.uint8, device=DEV), M * K
    a, b = blob(), blob()
    q4.q8_quantize(to_dev(bad), a)
    q4.q8_quantize(to_dev(x), b)
    check(q8_values(a, M, K), q8_values(b, M, K), nan, inf, 32, False)
    for bf16 in (False, True):
        for rows in (1, 128):
            out = []
            for v in (bad, x):
                q, s = torch.empty(n8, dtype=torch.uint8, device=DEV), torch.empty(-(-M // rows) * 4, device=DEV)
                (q4.f8_quantize_bf16 if bf16 else q4.f8_quantize)(dev_of(v, bf16), q, s, M, K, rows)
                out.append(f8_values(q, s, M, K, rows))
            if rows == 1:
                check(*out, nan, inf, 128, True)
            else:
                assert np.isnan(out[0][nan]).all() and not np.isfinite(out[0][inf]).any()


@pytest.mark.parametrize("gelu", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_activations(bf16, gelu):
    x, nan, inf = rows_with_faults(M, K)
    fn, tail = q4.Q4_ACT_GELU if gelu else q4.Q4_ACT_SILU, "_bf16" if bf16 else ""
    gate = np.abs(np.random.default_rng(4).normal(0, 1, (M, K))).astype(np.float32) + 0.5
    # The faults in the gate, then in the up half.
    for where in ("gate", "up"):
        g, u = gate.copy(), x.copy()
        (g if where == "gate" else u)[nan] = np.nan
        (g if where == "gate" else u)[inf] = np.inf
        vals = []
        for gv, uv in ((g, u), (gate, x)):
            blob, y = torch.empty(M * (K // 32) * 34, dtype=torch.uint8, device=DEV), torch.empty(M, K, device=DEV)
            q, s = torch.empty(M * K, dtype=torch.uint8, device=DEV), torch.empty(M * 4, device=DEV)
            gd, ud = dev_of(gv, bf16), dev_of(uv, bf16)
            getattr(q4, "q8_act" + tail)(gd, ud, blob, M, K, fn)
            getattr(q4, "f8_act" + tail)(gd, ud, q, s, M, K, fn)
            getattr(q4, "q4_act" + tail)(gd, ud, y, M, K, fn)
            want = torch.empty_like(q), torch.empty_like(s)
            q4.f8_quantize(y, *want, M, K, 1)
            v, w = f8_values(q, s, M, K), f8_values(*want, M, K)
            assert np.array_equal(v, w, equal_nan=True)
            vals.append((q8_values(blob, M, K), v))
        check(vals[0][0], vals[1][0], nan, inf, 32, False)
        check(vals[0][1], vals[1][1], nan, inf, 128, True)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("K,share", [(32, 1), (96, 3), (416, 1), (1056, 2), (4096, 1), (5120, 2), (11616, 1), (32768, 1)])
def test_norms(K, share, bf16):
    # Rows 1: a NaN in x; 2: in the residual; 3, 4: an infinity; 5: both signs of it in
    # one sum. The rows beside them are what they are without.
    M, tail = 7, "_bf16" if bf16 else ""
    g = np.random.default_rng(K)
    x, res = g.normal(0, 1, (M * share, K)).astype(np.float32), g.normal(0, 1, (M, K)).astype(np.float32)
    w = g.uniform(0.5, 1, (M, share)).astype(np.float32)
    bad_x, bad_r = x.copy(), res.copy()
    at = K - 2
    bad_x[1 * share, 3], bad_r[2, at] = np.nan, np.nan
    bad_x[4 * share - 1, 5], bad_r[4, at] = np.inf, -np.inf
    bad_x[5 * share, at], bad_r[5, at] = np.inf, -np.inf
    outs = []
    for xv, rv in ((bad_x, bad_r), (x, res)):
        sm = torch.empty(M, K, dtype=torch.bfloat16 if bf16 else torch.float32, device=DEV)
        y, y16 = torch.empty(M, K, device=DEV), torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
        blob = torch.empty(M * (K // 32) * 34, dtype=torch.uint8, device=DEV)
        q, s = torch.empty(M * K, dtype=torch.uint8, device=DEV), torch.empty(M * -(-K // 128), device=DEV)
        args, kw = (dev_of(xv, bf16), torch.ones(K, device=DEV)), dict(residual=dev_of(rv, bf16), weights=to_dev(w) if share > 1 else None, share=share)
        getattr(q4, "q4_norm" + tail)(*args, y, M, K, 1e-5, sum=sm, **kw)
        getattr(q4, "q4_norm" + tail)(*args, y16, M, K, 1e-5, **kw)
        getattr(q4, "q8_norm" + tail)(*args, blob, M, K, 1e-5, **kw)
        getattr(q4, "f8_norm" + tail)(*args, q, s, M, K, 1e-5, **kw)
        outs.append([t.float().cpu().numpy().astype(np.float64) for t in (sm, y, y16)] + [q8_values(blob, M, K), f8_values(q, s, M, K)])
    rest, other = [0, 6], np.arange(K)
    for got, clean in zip(*outs):
        assert np.array_equal(got[rest], clean[rest])
    sm, y, y16, v8, vf = outs[0]
    for v in (y, y16, v8, vf):
        assert np.isnan(v[[1, 2, 5]]).all()
        assert np.isnan(v[3, 5]) and np.isnan(v[4, at])
    for v in (y, y16, vf):
        assert (v[3, other != 5] == 0).all() and (v[4, other != at] == 0).all()
    assert np.isnan(sm[1, 3]) and np.isnan(sm[2, at]) and sm[3, 5] == np.inf and sm[4, at] == -np.inf and np.isnan(sm[5, at])
    for m, c in ((1, 3), (2, at), (3, 5), (4, at), (5, at)):
        assert np.isfinite(sm[m, other != c]).all()
