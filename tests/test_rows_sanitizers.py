"""Host code of the rows' way and of the MXFP4 calls under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only):
tests/sanitize/rows_driver.cpp with csrc/rows_abi.cpp, csrc/mx_abi.cpp, csrc/abi.cpp and the host stand-ins."""
import os
import shutil

import pytest

from tests.test_host_sanitizers import FLAGS, ROOT, SAN, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the HIP headers")
def test_rows_and_mx_host_code_under_sanitizers(tmp_path):
    exe = str(tmp_path / "rows_driver")
    csrc = os.path.join(ROOT, "quantized_moe_expert_topk_amd", "csrc")
    cmd = ["g++", "-std=c++17", *FLAGS, "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", csrc, *(os.path.join(csrc, f) for f in ("abi.cpp", "rows_abi.cpp", "mx_abi.cpp")),
           os.path.join(SAN, "host_stubs.cpp"), os.path.join(SAN, "rows_driver.cpp"), "-o", exe]
    assert "rows driver ok" in _build_and_run(cmd, exe, tmp_path)
