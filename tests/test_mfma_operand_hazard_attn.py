"""The compiled gfx950 code of the attention kernels keeps the distances between
matrix instructions and vector writes of their A and B registers that
tests/test_mfma_operand_hazard.py states for the GEMM kernels (its checks, on
these sources, with the flags that they are built with), holds no packed fp32
instruction, and leaves no kernel short of registers by more than the few values
that two workgroups on a CU cost.  Needs hipcc (skipped without it)."""
import os
import re
import shutil

import pytest

from nvfp4_w4a4_quantized_05_amd import build
from tests.test_mfma_operand_hazard import _closest_source_writes, _closest_source_writes_before


@pytest.fixture(scope="module", params=["nvfp4_attn_few.hip", "nvfp4_attn_many.hip"])
def listing(request, tmp_path_factory):
    hipcc = shutil.which("hipcc") or ("/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else None)
    if hipcc is None:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "attn.s"
    build.device_asm(request.param, str(out))
    return out.read_text()


def test_distances_around_matrix_instructions(listing):
    kern, kernels = None, {}
    for line in listing.splitlines():
        s = line.strip()
        m = re.match(r"^(_Z\S*):", s)
        if m:
            kern = m.group(1)
            kernels[kern] = []
        elif kern is not None and s and not s.startswith((".", ";", "//")) and not s.endswith(":"):
            kernels[kern].append(s.split(";")[0].strip())
    n = sum(s.startswith("v_mfma") for ins in kernels.values() for s in ins)
    assert n > 300, "no MFMA code found: the listing format changed"
    report = [f"{name[:60]}: `{mfma}` then `{valu}` ({d})" for name, ins in kernels.items()
              for d, mfma, valu in _closest_source_writes(ins)]
    report += [f"{name[:60]}: `{valu}` then `{mfma}` ({d})" for name, ins in kernels.items()
               for d, mfma, valu in _closest_source_writes_before(ins)]
    assert not report, "\n".join(report[:10])
    assert not any(s.startswith(("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32")) for ins in kernels.values() for s in ins)


def test_scratch_memory(listing):
    sizes = [int(x) for x in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", listing)]
    assert sizes and len(sizes) % 6 == 0  # three head sizes, two formats
    assert max(sizes) <= 128
