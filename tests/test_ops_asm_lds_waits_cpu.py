"""The tiled grouped products read LDS with inline-asm instructions and explicit
waits: on their gfx950 ISA, no instruction touches such a destination before a
wait that covers its read, on any control-flow path (the checker and its planted
mistake: test_asm_lds_waits_cpu.py)."""
import os
import subprocess

import pytest

from sparse_moe_layer_gemm_amd import build as pkg_build
from tests.test_asm_lds_waits_cpu import unsafe_asm_lds_reads

FILES = ["grouped_tile.hip", "grouped_stream.hip", "mxfp4_tile.hip"]


@pytest.mark.parametrize("src", FILES)
def test_inline_asm_lds_reads_complete_before_use(src, tmp_path):
    flags = [f for f in pkg_build.FLAGS if f != "-fPIC"]
    out = tmp_path / (src + ".s")
    r = subprocess.run([pkg_build.HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(pkg_build.CSRC, src),
                        "-o", str(out)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    text = out.read_text()
    n, bad = unsafe_asm_lds_reads(text)
    assert n > 0 and not bad, bad[:5]
    assert "scratch_load" not in text and "scratch_store" not in text  # nothing spills
