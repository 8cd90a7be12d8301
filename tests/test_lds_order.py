"""LDS that the lanes of one wavefront exchange without a workgroup barrier (CPU: read
from the sources). __builtin_amdgcn_wave_barrier touches no memory as the compiler
sees it, so that it alone does not keep one lane's store before another's load:
the fences around it do."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_weight_dequant_amd", "csrc")
BARRIER = "__builtin_amdgcn_wave_barrier()"
FENCED = re.compile(r'__builtin_amdgcn_fence\(__ATOMIC_RELEASE, "wavefront"\);\s*__builtin_amdgcn_wave_barrier\(\);\s*'
                    r'__builtin_amdgcn_fence\(__ATOMIC_ACQUIRE, "wavefront"\);')


def bare(text):
    return text.count(BARRIER) - len(FENCED.findall(text))


def test_the_rule_itself():
    fence = '__builtin_amdgcn_fence(__ATOMIC_%s, "wavefront");\n'
    assert bare(fence % "RELEASE" + BARRIER + ";\n" + fence % "ACQUIRE") == 0
    assert bare(BARRIER + ";") == 1
    assert bare(fence % "RELEASE" + BARRIER + ";\n") == 1


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "**", "*.h*"), recursive=True)), ids=os.path.basename)
def test_wave_barriers_are_fenced(path):
    assert bare(open(path).read()) == 0
