"""The waits of the weight gradient from kept rows, read in the compiled kernels."""
import os
import re
import subprocess

import pytest

from combine_get_dispatch_amd import build as epbuild


@pytest.mark.slow
def test_loads_behind_the_copies(tmp_path):
    """Before a step's barrier its copies to LDS are waited for by letting as many accesses be in flight as the step's first half
    has loads: there have to be so many, all after the last copy (a load moved, merged or left out would let a copy be late)."""
    out = str(tmp_path / "experts.s")
    subprocess.run([epbuild.hipcc()] + epbuild.flags() + ["-S", "--offload-device-only", "-o", out,
                   os.path.join(epbuild.CSRC, "ep_experts.hip")], check=True, capture_output=True)
    kernel, checked = "", {}
    lines = open(out).read().splitlines()
    for at, line in enumerate(lines):
        name = re.match(r"_ZN\S*k_wgradI(?:Li\d+E){4}Lb(\d)ELb(\d)E\S*:", line)
        if name:
            kernel = name.group(0) if name.group(2) == "1" else ""
            regions = name.group(1) == "1"
        if line.startswith("\t.section") or not kernel:
            kernel = kernel if not line.startswith("\t.section") else ""
            continue
        wait = re.match(r"\s*s_waitcnt vmcnt\((\d+)\) lgkmcnt\(0\)", line)
        if not wait or "s_barrier" not in lines[at + 1] or wait.group(1) == "0":
            continue
        loads, back = 0, at - 1
        while not re.search(r"s_barrier|global_load_lds|Loop Header", lines[back]):
            loads += bool(re.match(r"\s*global_load_(dwordx4|ubyte)\b", lines[back]))
            assert "s_cbranch" not in lines[back] or regions, lines[back]  # (regions: the look-up of rows, before the loads)
            back -= 1
        assert int(wait.group(1)) == 4
        assert loads >= int(wait.group(1)), f"{kernel}: {loads} loads before {line.strip()}"
        checked[kernel] = checked.get(kernel, 0) + 1
    assert len(checked) == 3 and all(n >= 1 for n in checked.values()), checked
