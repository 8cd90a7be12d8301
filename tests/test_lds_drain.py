"""Direct-to-LDS loads and the LDS stores that follow them, in the built library's
own gfx950 code (CPU: read with llvm-objdump).

A kernel that fills LDS rings by direct loads and then stores other data (the
partial tiles, the rows of y) over the rings must first wait until no load is
in flight, and meet the wavefronts that issued none: a load that lands later
overwrites what was stored. No run shows that reliably; the order of the instructions does."""
import os
import re
import shutil
import subprocess

import pytest

binding = pytest.importorskip("block_quantized_weight_dequant_amd.binding")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

needs_objdump = pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")


def events(asm):
    """Direct-to-LDS loads (L), vmcnt waits (their count), barriers (B) and LDS
    stores (S) of a kernel, in program order."""
    out = []
    for line in asm.splitlines():
        line = line.split("//")[0].strip()
        if line.startswith("buffer_load") and line.endswith(" lds"):
            out.append("L")
        elif line.startswith("s_waitcnt") and "vmcnt" in line:
            out.append(int(re.search(r"vmcnt\((\d+)\)", line).group(1)))
        elif line.startswith("s_barrier"):
            out.append("B")
        elif line.startswith("ds_write"):
            out.append("S")
    return out


def stores_into_flying_loads(ev):
    """LDS stores behind a direct load whose last counted barrier let loads fly."""
    loaded, drained, wait, bad = False, False, None, 0
    for e in ev:
        if e == "L":
            loaded, drained, wait = True, False, None
        elif e == "B":
            # A barrier without a wait of its own changes nothing.
            drained = drained if wait is None else wait == 0
            wait = None
        elif e == "S":
            bad += loaded and not drained
        else:
            wait = e
    return bad


def test_the_rule_itself():
    assert stores_into_flying_loads(["L", 25, "B", "S"]) == 1
    assert stores_into_flying_loads(["L", 0, "B", 25, "B", "S"]) == 1     # the branch that counts is the later one
    assert stores_into_flying_loads(["L", 25, "B", 0, "B", "S", "B", "S"]) == 0
    assert stores_into_flying_loads(["S", "B", "L", 0, "S"]) == 1          # no meeting
    assert stores_into_flying_loads(["S", 3, "B"]) == 0


@needs_objdump
def test_rings_are_drained_before_their_lds_is_stored_to(tmp_path):
    lib = shutil.copy(binding.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, capture_output=True, check=True)
    seen = {}
    for f in os.listdir(tmp_path):
        if not f.endswith("gfx950"):
            continue
        dis = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", os.path.join(tmp_path, f)],
                             capture_output=True, text=True, check=True).stdout
        for part in re.split(r"\n(?=<)", dis):
            name = re.match(r"<(\S+)>:", part)
            ev = events(part) if name else []
            if "L" in ev:
                seen[name.group(1)] = stores_into_flying_loads(ev)
    # Every kernel that has such loads, the GEMM's and the grouped products' among them.
    for kernel in ("k_gemm_split", "k_gemm_split_grouped", "k_grouped_few", "k_f8_rows", "k_f8_rows_grouped", "k_f8_tile"):
        assert any("%d%sI" % (len(kernel), kernel) in n for n in seen), kernel
    assert not {n: v for n, v in seen.items() if v}
