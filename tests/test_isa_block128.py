"""The block-128 kernels as built: no scratch access in a K loop, and no spills."""

from test_isa import _loops, code_objects, disasm_text, kernel_spills  # noqa: F401


def test_no_scratch_access_inside_k_loops(disasm_text):  # noqa: F811
    """The innermost loops with MFMAs, that is, without a tile's stores."""
    seen = 0
    for name, body in _loops(disasm_text, "block128_"):
        if not any(i.startswith("v_mfma") for i in body) or any("_store_" in i for i in body if not i.startswith("scratch")):
            continue
        seen += 1
        bad = [i for i in body if i.startswith("scratch_")]
        assert not bad, f"{name}: scratch access in a K loop: {bad[:2]}"
    assert seen >= 40, "fewer K loops than the instances hold"


def test_no_spills(kernel_spills):  # noqa: F811
    kernels = {k: v for k, v in kernel_spills.items() if "block128_" in k}
    assert len(kernels) >= 80
    assert all(v == 0 for v in kernels.values()), {k: v for k, v in kernels.items() if v}
