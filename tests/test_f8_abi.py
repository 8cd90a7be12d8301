"""CPU tests of the E4M3 entry points (include/f8.h): declared and exported
symbols agree, and every invalid argument is refused before a launch."""
import os
import re
import subprocess

import pytest

from test_abi import A, ROOT, W, Y, fake_addresses

binding = pytest.importorskip("block_quantized_weight_dequant_amd.binding")
S = binding
HEADER = os.path.join(ROOT, "include", "f8.h")
AS, WS = A + (1 << 28), W + (1 << 28)


def test_exports_match_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))
    assert declared == sorted(binding.F8_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert sorted(l.split()[-1] for l in out.splitlines() if l.split()[-1].startswith("f8_")) == declared
    defs = {k: int(v) for k, v in re.findall(r"#define\s+(F8_\w+)\s+(\d+)", text)}
    assert defs == {"F8_BLOCK": binding.F8_BLOCK, "F8_MAX_K": binding.F8_MAX_K}


def _codec(entry, x, M, K, br, q, qb, s, se, extra=None):
    if entry == "f8_dequant":
        return binding.raw_status(entry, q, qb, s, se, M, K, br, x, M * K if extra is None else extra, 0)
    return binding.raw_status(entry, x, M, K, br, q, qb, s, se, 0)


@fake_addresses
@pytest.mark.parametrize("entry", ["f8_quantize", "f8_quantize_bf16", "f8_dequant"])
def test_codec_argument_checks(entry):
    st = lambda *a, **k: _codec(entry, *a, **k)
    for M, K, br in [(-1, 64, 1), (4, 0, 1), (4, 48, 1), (4, -32, 1), (4, 64, 2), (4, 64, 0)]:
        assert st(A, M, K, br, W, 256, Y, 4, extra=256) == S.Q4_ERR_SHAPE, (M, K, br)
    assert st(A, 4, 160, 1, W, 639, Y, 8) == S.Q4_ERR_SIZE
    assert st(A, 4, 160, 1, W, 640, Y, 4) == S.Q4_ERR_SIZE
    assert st(A, 4, 160, 128, W, 640, Y, 8) == S.Q4_ERR_SIZE      # two tiles, not eight blocks
    assert st(A, 2 ** 31 - 1, 160, 1, W, (2 ** 31 - 1) * 160, Y, 2 * (2 ** 31 - 1)) == S.Q4_ERR_SIZE
    assert st(None, 0, 160, 1, None, 0, None, 0) == S.Q4_OK
    for x, q, s in [(None, W, Y), (A, None, Y), (A, W, None)]:
        assert st(x, 4, 160, 1, q, 640, s, 8) == S.Q4_ERR_NULL
    for x, q, s in [(A + 8, W, Y), (A, W + 8, Y), (A, W, Y + 4)]:
        assert st(x, 4, 160, 1, q, 640, s, 8) == S.Q4_ERR_ALIGN
    assert st(A, 4, 160, 1, A + 16, 640, Y, 8) == S.Q4_ERR_ALIAS
    assert st(A, 4, 160, 1, W, 640, A + 16, 8) == S.Q4_ERR_ALIAS
    if entry != "f8_dequant":    # its two outputs apart; f8_dequant only reads them
        assert st(A, 4, 160, 1, W, 640, W + 624, 8) == S.Q4_ERR_ALIAS
    else:
        assert st(A, 4, 160, 1, W, 640, Y, 8, extra=639) == S.Q4_ERR_SIZE


@fake_addresses
@pytest.mark.parametrize("entry", ["f8_gemm", "f8_gemv"])
def test_product_argument_checks(entry):
    st = lambda a, a_s, w, wb, w_s, y, M, N, K: binding.raw_status(entry, a, a_s, w, wb, w_s, y, M, N, K, 0)
    for M, N, K in [(-1, 4, 64), (1, -4, 64), (1, 4, 48), (1, 4, 0), (1, 4, F(1) + 32)]:
        assert st(A, AS, W, 4 * K, WS, Y, M, N, K) == S.Q4_ERR_SHAPE, (M, N, K)
    assert st(A, AS, W, 255, WS, Y, 1, 4, 64) == S.Q4_ERR_SIZE
    assert st(None, None, None, 256, None, None, 0, 4, 64) == S.Q4_OK
    assert st(None, None, None, 0, None, None, 4, 0, 64) == S.Q4_OK
    ok = [A, AS, W, 256, WS, Y]
    for i in (0, 1, 2, 4, 5):
        assert st(*[None if j == i else v for j, v in enumerate(ok)], 2, 4, 64) == S.Q4_ERR_NULL
        assert st(*[v + 8 if j == i else v for j, v in enumerate(ok)], 2, 4, 64) == S.Q4_ERR_ALIGN
        if i != 5:
            assert st(*ok[:5], ok[i], 2, 4, 64) == S.Q4_ERR_ALIAS
    # y is two bytes an element: [2, 8] spans 32 bytes.
    assert st(Y + 16, AS, W, 512, WS, Y, 2, 8, 64) == S.Q4_ERR_ALIAS


def F(n):
    return n * binding.F8_MAX_K


@fake_addresses
def test_gemv_row_limit():
    assert binding.raw_status("f8_gemv", A, AS, W, 256, WS, Y, 9, 4, 64, 0) == S.Q4_ERR_SHAPE
