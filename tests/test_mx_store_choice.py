"""When the values of quantised rows are stored past the caches (csrc/tiles.h on the CPU): bf16 in rows of whole 128-byte lines,
which a wave writes whole.  Never fp32: a wave's two stores write 16 of every 32 bytes each, and lines written in parts take up
to twice as long (8192 x 4096: 58 us, through the caches 36)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the HIP headers")
    so = str(tmp_path_factory.mktemp("stores") / "mx_store_choice.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__",
                    "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "quantized_moe_expert_topk_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host", "mx_store_choice.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    return lambda y, K, f32: lib.values_non_temporal(ctypes.c_uint64(y), K, f32)


@pytest.mark.parametrize("K", [32, 64, 96, 1024, 4096, 8192])
def test_values(choice, K):
    assert choice(1 << 40, K, 0) == (K % 64 == 0)
    assert choice((1 << 40) + 64, K, 0) == 0
    assert choice(1 << 40, K, 1) == 0
