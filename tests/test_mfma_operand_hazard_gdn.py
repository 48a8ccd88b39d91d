"""The compiled gfx950 code of the chunked Gated DeltaNet kernels keeps the
distances between matrix instructions and vector writes of their A and B
registers that tests/test_mfma_operand_hazard.py states for the GEMM kernels
(its checks, on this source).  Needs hipcc (skipped without it)."""
import os
import re
import shutil
import subprocess

import pytest

from tests.conftest import ROOT
from tests.test_mfma_operand_hazard import _closest_source_writes, _closest_source_writes_before


@pytest.fixture(scope="module")
def chunk_kernels_asm(tmp_path_factory):
    hipcc = shutil.which("hipcc") or ("/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else None)
    if hipcc is None:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "chunk.s"
    src = os.path.join(ROOT, "nvfp4_w4a4_quantized_05_amd", "csrc", "nvfp4_gdn_chunk.hip")
    cmd = [hipcc, "-O3", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-mllvm", "-pragma-unroll-threshold=1000000", "-I", os.path.join(ROOT, "include"),
           "--cuda-device-only", "-S", "-o", str(out), src]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    kern, kernels = None, {}
    for line in out.read_text().splitlines():
        s = line.strip()
        m = re.match(r"^(_Z\S*):", s)
        if m:
            kern = m.group(1)
            kernels[kern] = []
        elif kern is not None and s and not s.startswith((".", ";", "//")) and not s.endswith(":"):
            kernels[kern].append(s.split(";")[0].strip())
    return kernels


def test_distances_around_matrix_instructions(chunk_kernels_asm):
    n = sum(s.startswith("v_mfma") for ins in chunk_kernels_asm.values() for s in ins)
    assert n > 300, "no MFMA code found: the listing format changed"
    report = [f"{name[:60]}: `{mfma}` then `{valu}` ({d})" for name, ins in chunk_kernels_asm.items()
              for d, mfma, valu in _closest_source_writes(ins)]
    report += [f"{name[:60]}: `{valu}` then `{mfma}` ({d})" for name, ins in chunk_kernels_asm.items()
               for d, mfma, valu in _closest_source_writes_before(ins)]
    assert not report, "\n".join(report[:10])
    assert not any("v_pk_" in s and "_f32" in s and not s.startswith("v_cvt") for ins in chunk_kernels_asm.values() for s in ins)
