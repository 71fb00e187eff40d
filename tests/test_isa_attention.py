"""Properties of the compiled attention kernels (CPU only: hipcc cross-compiles for gfx950).

Their working arrays (queries, running outputs, codes on their way) live in registers as long as every
index into them is a constant once loops are written out.  Where the compiler leaves one loop as it is, the
arrays move to scratch memory and the results stay right, many times slower.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from rotation_w4a4_quantized_convrot_amd import build as B


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("isa") / "kv8.s")
    cmd = [hipcc, *B.HIPCC_FLAGS, "-I", B.INCLUDE, "-I", B.CSRC, "--cuda-device-only", "-S",
           os.path.join(B.CSRC, "kv8.hip"), "-o", out]
    done = subprocess.run(cmd, check=True, capture_output=True, text=True)
    with open(out) as f:
        return f.read(), done.stderr


@pytest.mark.parametrize("kernel,forms", [("few_rows_kernel", 18), ("many_rows_kernel", 6)])
def test_attention_uses_no_scratch(compiled, kernel, forms):
    """Every form: both input types, heads up to 64, 128 and 256, and the tiles of rows."""
    text, _ = compiled
    names = [n for n in re.findall(r"^(_Z\S+):", text, re.M) if kernel in n]
    assert len(names) == forms
    for name in names:
        end = text.index(".Lfunc_end", text.index(name + ":"))
        scratch = int(re.search(r"ScratchSize:\s*(\d+)", text[end:end + 4000]).group(1))
        assert scratch == 0, f"{name}: {scratch} bytes of scratch per lane"


def test_every_loop_is_written_out(compiled):
    _, warnings = compiled
    assert "not unrolled" not in warnings, warnings
