"""Scalar registers that the block-128 kernels spill (to lanes of vector registers, never to memory), as built."""

import re
import subprocess

import pytest

from test_isa import _tool, code_objects  # noqa: F401

# The most that a kernel of each form spills: the plain product in its 64 x 128 tiles; with an end and by expert along the rows,
# whose tile ends read the pointers and row distances of up to five tensors; by expert along K.
MOST = {"0": 13, "1": 39, "2": 65, "3": 0}


@pytest.fixture(scope="module")
def scalar_spills(code_objects):  # noqa: F811
    readelf = _tool("llvm-readelf")
    if not readelf:
        pytest.skip("llvm-readelf not found")
    spills = {}
    for code in code_objects:
        notes = subprocess.run([readelf, "--notes", code], check=True, capture_output=True, text=True).stdout
        for kernel in notes.split("  - .")[1:]:
            name, count = re.search(r"\.name:\s+(\S+)", kernel), re.search(r"\.sgpr_spill_count:\s+(\d+)", kernel)
            if name and count:
                spills[name.group(1)] = int(count.group(1))
    return spills


def test_scalar_spills(scalar_spills):
    most = {form: 0 for form in MOST}
    others = 0
    for name, count in scalar_spills.items():
        if "block128_" not in name:
            continue
        form = re.search(r"FormE(\d)", name)
        if form:
            most[form.group(1)] = max(most[form.group(1)], count)
        else:
            others = max(others, count)
    assert others == 0 and all(most[f] <= MOST[f] for f in MOST), (others, most)
