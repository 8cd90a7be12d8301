"""The library's own rules for which kernel a product takes (csrc/f8_forms.h,
csrc/validate.h: plain C++), compiled by the host compiler, so that tests can
hold their cases to the kernels they are meant for."""
import ctypes
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "f8_forms.h"
#include "validate.h"
extern "C" {
int f8(int M, int N) { const q4v::F8Choice c = q4v::f8_form(M, N); return c.form * 8 + c.rg; }
int f8_grouped(int G, int M, int N) { const q4v::F8Choice c = q4v::f8_form_grouped(G, M, N); return c.form * 8 + c.rg; }
int grouped(int G, int M, int N, int K, int block_bytes, int a_elem)
{
    if (q4v::grouped_in_place(M, N, K, (size_t)block_bytes, (size_t)a_elem)) return 0;
    if (!q4v::grouped_few(G, M, N, K)) return 1;
    const q4v::FewShape f = q4v::grouped_few_shape(G, M, N, (size_t)block_bytes);
    return 16 * f.ct + f.r;
}
}
"""
_lib = None


def _load():
    global _lib
    if _lib is None:
        with tempfile.TemporaryDirectory() as d:
            src, out = os.path.join(d, "forms.cpp"), os.path.join(d, "forms.so")
            with open(src, "w") as f:
                f.write(SOURCE)
            subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                            "-I" + os.path.join(ROOT, "block_quantized_weight_dequant_amd", "csrc"), src, "-o", out], check=True)
            _lib = ctypes.CDLL(out)
    return _lib


TILES = ("quarter", "half", "small", "wide", "large")


def _f8_name(c):
    return "rows%d" % (c % 8) if c < 8 else TILES[c // 8 - 1]


def f8(M, N):
    """rows1 .. rows4 (row groups), or a tile's name."""
    return _f8_name(_load().f8(M, N))


def f8_grouped(G, M, N):
    return _f8_name(_load().f8_grouped(G, M, N))


def grouped(G, M, N, K, fmt, act):
    """in place, few<weight rows / 16>x<row subtiles>, or tiles."""
    c = _load().grouped(G, M, N, K, {"q4": 18, "q8": 34}[fmt], {"f32": 4, "bf16": 2}[act])
    return "in place" if c == 0 else "tiles" if c == 1 else "few%dx%d" % (c // 16, c % 16)
