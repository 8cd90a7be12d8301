"""CPU tests of the router's and the grouped products' argument checks and
workspace sizes (include/q4.h, include/f8.h)."""
import pytest

from test_abi import A, W, Y, fake_addresses

binding = pytest.importorskip("block_quantized_weight_dequant_amd.binding")
S = binding
AS, WS, OFF, ORD, WORK = A + (1 << 28), W + (1 << 30), Y + (1 << 32), Y + (2 << 32), Y + (3 << 32)
GROUPED = [(f, act) for f in ("q4", "q8") for act in ("", "_bf16")]
BYTES = {"q4": 18, "q8": 34}


def test_constants_match_header():
    import re
    from test_abi import HEADER
    defs = dict(re.findall(r"#define\s+(Q4_MAX_\w+)\s+(\d+)", open(HEADER).read()))
    assert {k: int(v) for k, v in defs.items()} == {
        "Q4_MAX_EXPERTS": S.Q4_MAX_EXPERTS, "Q4_MAX_TOP_K": S.Q4_MAX_TOP_K, "Q4_MAX_SLOTS": S.Q4_MAX_SLOTS}


def test_route_workspace_bytes():
    f = binding.q4_route_workspace_bytes
    for T in (0, 1, 64):
        assert f(T, 8, 2) == 0
    assert f(65, 8, 2) == 3 * 8 * 4            # chunks of 32 tokens
    assert f(8192, 64, 6) == 256 * 64 * 4
    assert f(8193, 64, 6) == 249 * 64 * 4      # chunks of 33
    for T, E, k in [(-1, 8, 2), (100, 0, 1), (100, 1025, 2), (100, 8, 9), (100, 8, 0), (100, 64, 33), (2 ** 30, 8, 2)]:
        assert f(T, E, k) == 0


@fake_addresses
def test_route_argument_checks():
    ok = dict(x=A, ids=W, wt=W + (1 << 20), off=OFF, order=ORD, ws=WORK, wsb=1 << 20)

    def st(T=100, E=8, k=2, **kw):
        a = {**ok, **kw}
        return binding.raw_status("q4_route", a["x"], T, E, k, 1, a["ids"], a["wt"], a["off"], a["order"], a["ws"], a["wsb"], 0)

    for T, E, k in [(-1, 8, 2), (100, 0, 1), (100, 1025, 2), (100, 8, 9), (100, 8, 0), (100, 64, 33), (2 ** 30, 8, 2)]:
        assert st(T, E, k) == S.Q4_ERR_SHAPE, (T, E, k)
    assert binding.raw_status("q4_route", None, 0, 8, 2, 1, None, None, None, None, None, 0, 0) == S.Q4_OK
    for name in ("x", "ids", "wt", "off", "order"):
        assert st(**{name: None}) == S.Q4_ERR_NULL
        assert st(**{name: ok[name] + 4}) == S.Q4_ERR_ALIGN
        for other in ("x", "ids", "wt", "off", "order"):
            if other != name:
                assert st(**{name: ok[other] + 16}) == S.Q4_ERR_ALIAS, (name, other)
    need = binding.q4_route_workspace_bytes(100, 8, 2)
    assert st(wsb=need - 1) == S.Q4_ERR_WORKSPACE
    assert st(ws=None) == S.Q4_ERR_NULL
    assert st(ws=WORK + 8) == S.Q4_ERR_ALIGN
    assert st(ws=A + 16) == S.Q4_ERR_ALIAS
    assert st(ws=ORD - 64) == S.Q4_ERR_ALIAS


@pytest.mark.parametrize("f,act", GROUPED)
def test_grouped_workspace_bytes(f, act):
    ws = getattr(binding, f + "_gemm_grouped" + act + "_workspace_bytes")
    e = 2 if act else 4
    pad = lambda n: -(-n // 256) * 256
    for M in range(1, 9):
        assert ws(8, M, 64, 4096) == 0                                            # multiplied in place
    assert ws(8, 9, 64, 4096) == pad(8 * 16 * 4) + 8 * 16 * 4096 * e              # eight 16-row tiles at most
    big = 2 ** 31 // (8 * BYTES[f])                                               # the first N whose W[e] reaches 2^31 bytes
    assert ws(8, 2, big, 256) == 0
    assert ws(8, 2, big + 1, 256) == pad(2 * 16 * 4) + 2 * 16 * 256 * e
    assert ws(8, 256, 64, 4096) == pad(24 * 16 * 4) + 24 * 16 * 4096 * e
    assert ws(8, 257, 14336, 4096) == pad(24 * 16 * 4) + 24 * 16 * 4096 * e
    assert ws(8, 400, 14336, 4096) == pad(11 * 128 * 4) + 11 * 128 * 4096 * e     # more rows of many columns: 128-row tiles
    assert ws(8, 400, 64, 4096) == pad(33 * 16 * 4) + 33 * 16 * 4096 * e          # of few columns
    assert ws(1, 2 ** 19 + 128, 64, 64) == pad(4098 * 128 * 4) + 4098 * 128 * 64 * e
    assert ws(8, 2, 64, 64) == pad(2 * 16 * 4) + 2 * 16 * 64 * e                  # K % 256 != 0: not in place
    assert ws(8, 9, 64, 14336) == pad(8 * 16 * 4) + 8 * 16 * 14336 * e
    assert ws(8, 9, 64, 14592) == pad(8 * 128 * 4) + 8 * 128 * 14592 * e          # past 112 blocks a wavefront: 128-row tiles
    for G, M, N, K in [(0, 2, 4, 64), (1025, 2, 4, 64), (8, 0, 4, 64), (8, -1, 4, 64), (8, 2, 0, 64), (8, 2, 4, 32),
                       (8, 2, 4, 96), (8, 2, 4, 2 ** 22 + 64), (8, 2 ** 30 + 1, 4, 64)]:
        assert ws(G, M, N, K) == 0, (G, M, N, K)


def _grouped_args(f, act):
    G, M, N, K, share = 3, 8, 16, 128, 2
    need = getattr(binding, f + "_gemm_grouped" + act + "_workspace_bytes")(G, M, N, K)
    return dict(a=A, w=W, wb=G * N * (K // 32) * BYTES[f], off=OFF, order=ORD, share=share, y=Y, G=G, M=M, N=N, K=K,
                ws=WORK, wsb=need)


@fake_addresses
@pytest.mark.parametrize("f,act", GROUPED)
def test_grouped_argument_checks(f, act):
    ok = _grouped_args(f, act)

    def st(**kw):
        v = {**ok, **kw}
        return binding.raw_status(f + "_gemm_grouped" + act, v["a"], v["w"], v["wb"], v["off"], v["order"], v["share"], v["y"],
                                  v["G"], v["M"], v["N"], v["K"], v["ws"], v["wsb"], 0)

    for kw in [dict(G=0), dict(G=1025), dict(M=-1), dict(M=2 ** 30 + 1), dict(N=-1), dict(K=0), dict(K=96), dict(K=2 ** 22 + 64),
               dict(share=0)]:
        assert st(**kw) == S.Q4_ERR_SHAPE, kw
    assert st(wb=ok["wb"] - 1) == S.Q4_ERR_SIZE
    assert st(G=2) == S.Q4_ERR_SIZE
    assert st(M=0, a=None, w=None, off=None, y=None, ws=None) == S.Q4_OK
    assert st(N=0, wb=0, a=None, w=None, off=None, y=None, ws=None) == S.Q4_OK
    for name in ("a", "w", "off", "y"):
        assert st(**{name: None}) == S.Q4_ERR_NULL
    for name in ("a", "w", "off", "order", "y", "ws"):
        assert st(**{name: ok[name] + 8}) == S.Q4_ERR_ALIGN
    for name in ("a", "w", "off", "order"):
        assert st(y=ok[name]) == S.Q4_ERR_ALIAS
        assert st(ws=ok[name]) == S.Q4_ERR_ALIAS
    assert st(ws=Y + 256) == S.Q4_ERR_ALIAS
    # a is [ceil(M / share), K]: y right behind it does not overlap.
    end = A + 4 * 128 * (2 if act else 4)
    assert st(y=end, wsb=0) == S.Q4_ERR_WORKSPACE and st(y=end, share=1, wsb=0) == S.Q4_ERR_ALIAS
    assert st(order=None, wsb=0) == S.Q4_ERR_WORKSPACE     # no order: every other check passed
    assert st(wsb=ok["wsb"] - 1) == S.Q4_ERR_WORKSPACE
    assert st(ws=None) == S.Q4_ERR_NULL


@fake_addresses
def test_f8_grouped_argument_checks():
    ok = dict(a=A, a_s=AS, w=W, wb=3 * 16 * 160, w_s=WS, off=OFF, order=ORD, share=2, y=Y, G=3, M=8, N=16, K=160)

    def st(**kw):
        v = {**ok, **kw}
        return binding.raw_status("f8_gemm_grouped", *(v[k] for k in ("a", "a_s", "w", "wb", "w_s", "off", "order", "share", "y",
                                                                      "G", "M", "N", "K")), 0)

    for kw in [dict(G=0), dict(G=1025), dict(M=-1), dict(M=2 ** 30 + 1), dict(N=-1), dict(K=0), dict(K=48),
               dict(K=2 ** 22 + 32), dict(share=0), dict(M=2 ** 26, share=1, K=32), dict(M=2 ** 27 - 1, K=32, share=2)]:
        assert st(**kw) == S.Q4_ERR_SHAPE, kw
    assert st(wb=ok["wb"] + 1) == S.Q4_ERR_SIZE
    assert st(M=0, a=None, w=None, off=None, y=None) == S.Q4_OK
    assert st(N=0, wb=0, a=None, w=None, off=None, y=None) == S.Q4_OK
    for name in ("a", "a_s", "w", "w_s", "off", "y"):
        assert st(**{name: None}) == S.Q4_ERR_NULL
        assert st(**{name: ok[name] + 8}) == S.Q4_ERR_ALIGN
        if name != "y":
            assert st(y=ok[name]) == S.Q4_ERR_ALIAS
    assert st(order=ORD + 4) == S.Q4_ERR_ALIGN and st(y=ORD) == S.Q4_ERR_ALIAS
