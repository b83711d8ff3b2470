"""Inline assembly tells the compiler every register it writes (CPU only: reads the sources and cross-compiles)."""
import glob
import os
import re

from test_kernel_isa import _device_asm, pytestmark  # noqa: F401

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dequant_iqk_moe_amd", "csrc")


def _statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
            depth, i, quoted = 1, m.end(), False
            while depth:
                c = text[i]
                if c == '"' and text[i - 1] != "\\":
                    quoted = not quoted
                elif not quoted:
                    depth += (c == "(") - (c == ")")
                i += 1
            yield os.path.basename(path), text[m.start():i]


def test_m0_is_named_where_it_is_written():
    writers = [(f, s) for f, s in _statements() if re.search(r"\bs_mov_b32 m0\b", s)]
    assert writers
    for f, s in writers:
        assert '"m0"' in s.rsplit(":", 1)[1], (f, s)


def test_nothing_else_uses_m0(tmp_path):
    """Each setting of m0 in the tile kernels is followed at once by the copy it is for."""
    lines = [l.split(";")[0].strip() for l in _device_asm("iqk_fp8_tile.hip", tmp_path).splitlines()]
    lines = [l for l in lines if l and not l.startswith((".", "//"))]
    at = [i for i, l in enumerate(lines) if re.search(r"\bm0\b", l)]
    assert at
    for i in at:
        assert lines[i].startswith("s_mov_b32 m0, s") and lines[i + 1] == "s_nop 0", lines[i:i + 3]
        assert lines[i + 2].startswith("global_load_lds_dword"), lines[i:i + 3]
