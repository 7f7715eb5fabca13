"""The scan's loads of whole rows of states on the CPU: tests/c/scan_runs.cpp, which builds the kernels' own
header for the host under AddressSanitizer (host code alone; nothing is built for the GPU)."""

import os

import pytest

from test_sanitizers import C_DIR, ROOT, _build_and_run

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_runs_stay_in_their_rows(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not found")
    exe = str(tmp_path / "scan_runs")
    cmd = [HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-g", "-Xarch_host", "-fsanitize=address",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(ROOT, 'causal_conv1d_verify_amd', 'csrc')}",
           os.path.join(C_DIR, "scan_runs.cpp"), "-o", exe]
    out = _build_and_run(cmd, exe)
    assert "256 runs" in out
