"""The kernels around the routed experts run from registers and LDS alone, and
nothing else uses m0 where copies into LDS set it (CPU only: hipcc
cross-compiles)."""
import re

import pytest

from test_kernel_isa import _device_asm, _kernels, pytestmark  # noqa: F401


@pytest.mark.parametrize("src", ["iqk_sort.hip", "iqk_norm.hip", "iqk_int8_rows.hip", "iqk_int8_tile.hip"])
def test_no_scratch(src, tmp_path):
    asm = _device_asm(src, tmp_path)
    _, meta = _kernels(asm)
    assert meta, "no kernels found"
    for name, m in meta.items():
        assert m.get("private_segment_fixed_size", 0) == 0, name
        assert m.get("vgpr_spill_count", 0) == 0, name
    lines = [l.split(";")[0].strip() for l in asm.splitlines()]
    lines = [l for l in lines if l and not l.startswith((".", "//"))]
    at = [i for i, l in enumerate(lines) if re.search(r"\bm0\b", l)]
    assert bool(at) == (src == "iqk_int8_tile.hip")
    for i in at:
        assert lines[i].startswith("s_mov_b32 m0, s") and lines[i + 1] == "s_nop 0", lines[i:i + 3]
        assert re.match(r"buffer_load_dwordx4 .* lds$", lines[i + 2]), lines[i:i + 3]
