"""CPU sanitizer leg of libseqops.so's host side: sq_api.cpp built by g++ with AddressSanitizer and
UndefinedBehaviorSanitizer, stand-ins for the kernels' pickers and the HIP runtime (nothing here is
built for the GPU), and tests/c/sq_abi_sanitize.cpp's fuzz of shapes over the full range of every
field: a refused call launches nothing, an accepted one launches the grids that its plan needs within
the hardware's limits, and rows cut into segments fit the grid and the workspace."""

import os

import pytest

from test_sanitizers import C_DIR, ROOT, SAN, _build_and_run, _need


def test_sequence_ops_host_code_under_asan_ubsan(tmp_path):
    _need("g++")
    hip_inc = "/opt/rocm/include"
    if not os.path.exists(os.path.join(hip_inc, "hip", "hip_runtime_api.h")):
        pytest.skip("HIP headers not found")
    exe = str(tmp_path / "sq_abi_sanitize")
    csrc = os.path.join(ROOT, "causal_conv1d_verify_amd", "csrc")
    cmd = ["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", f"-I{hip_inc}", f"-I{os.path.join(ROOT, 'include')}",
           f"-I{csrc}", os.path.join(csrc, "sq_api.cpp"), os.path.join(C_DIR, "sq_abi_sanitize.cpp"), "-o", exe]
    out = _build_and_run(cmd, exe, ["600000"])
    assert "fuzz: 600000 shapes" in out
