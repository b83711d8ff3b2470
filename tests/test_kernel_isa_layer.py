"""The selection and 8-bit kernels run from registers and LDS alone (CPU only:
hipcc cross-compiles)."""
import pytest

from test_kernel_isa import _device_asm, _kernels, pytestmark  # noqa: F401


@pytest.mark.parametrize("src", ["iqk_router.hip", "iqk_fp8_prep.hip", "iqk_fp8_rows.hip", "iqk_fp8_tile.hip"])
def test_no_scratch(src, tmp_path):
    _, meta = _kernels(_device_asm(src, tmp_path))
    assert meta, "no kernels found"
    for name, m in meta.items():
        assert m.get("private_segment_fixed_size", 0) == 0, name
        assert m.get("vgpr_spill_count", 0) == 0, name
