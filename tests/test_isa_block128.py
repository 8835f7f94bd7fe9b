"""The block-128 product's kernels as built: no scratch access in a K loop, and none at all in the kernels of one scale per
column block."""

from test_isa import _loops, code_objects, disasm_text, kernel_spills  # noqa: F401


def test_no_scratch_access_inside_k_loops(disasm_text):  # noqa: F811
    """The innermost loops with MFMAs, that is, without a tile's stores."""
    seen = 0
    for name, body in _loops(disasm_text, "block128_"):
        if not any(i.startswith("v_mfma") for i in body) or any(i.startswith("buffer_store") for i in body):
            continue
        seen += 1
        bad = [i for i in body if i.startswith("scratch_")]
        assert not bad, f"{name}: scratch access in a K loop: {bad[:2]}"
    assert seen >= 40, "fewer K loops than the instances hold"


def test_no_spills_but_with_a_scale_per_column(kernel_spills):  # noqa: F811
    """block128_{tile,exact}_kernel<TileShape<...>, FA, FB, (CT,) BROWS>: with BROWS the 256 x 256 tile, whose accumulators
    take half of the registers, keeps 16 scales more and spills what only its tile end uses."""
    plain = {k: v for k, v in kernel_spills.items() if "block128_" in k and "Lb1EEEv" not in k}
    assert len(plain) >= 40
    assert all(v == 0 for v in plain.values()), {k: v for k, v in plain.items() if v}
