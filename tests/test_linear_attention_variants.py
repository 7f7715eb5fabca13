"""Which kernel a call gets, asked of the library (host only): the rules on both sides of their
borders, and the launches of the shapes that are timed."""

import ctypes
import os
import subprocess

import pytest

from causal_conv1d_verify_amd import _lib as base
from causal_conv1d_verify_amd import _linattn as la

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = base.CV_BF16, base.CV_F32
PREFILL, UPDATE, VERIFY, COMMIT = la.LA_CALL_PREFILL, la.LA_CALL_UPDATE, la.LA_CALL_VERIFY, la.LA_CALL_COMMIT
TOKENS, FEW, CHUNKED, CHUNKED_F32 = (la.LA_KERNEL_TOKENS, la.LA_KERNEL_FEW, la.LA_KERNEL_CHUNKED,
                                     la.LA_KERNEL_CHUNKED_F32)


def _shape(n_seq, T, hq, hv, dk=128, dv=128, x=BF16, state=F32, tokens=0, far=0):
    q, v = far or hq * dk, far or hv * dv
    return la.LaShape(n_seq, T, hq, hv, dk, dv, 0.1, x, state, n_seq, T * q, q, dk, T * q, q, dk, T * v, v, dv,
                      T * v, v, dv, T * hv, hv, hv * dk * dv, tokens)


def _info(call, shape):
    if not os.path.exists(la.LIB_PATH):
        pytest.skip("liblinattn.so not built (run __graft_entry__.build())")
    lib, info = la.load(), la.LaLaunchInfo()
    rc = lib.linattn_describe(call, shape, ctypes.byref(info))
    assert rc == 0, lib.linattn_last_error()
    if call == PREFILL:
        assert info.workspace_bytes == lib.linattn_prefill_workspace(shape)
        assert (info.segment_tokens > 0) == (info.launches == 3) == (info.workspace_bytes > 0)
    return info


def test_struct_layout(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "linear_attention.h"\nint main(void) {\n'
                   'printf("%zu", sizeof(la_launch_info_t));\n' +
                   "".join(f'printf(" %zu", offsetof(la_launch_info_t, {n}));\n' for n, _ in la.LaLaunchInfo._fields_) +
                   "".join(f'printf(" %d", {n});\n' for n in (
                       "LA_CALL_PREFILL", "LA_CALL_UPDATE", "LA_CALL_VERIFY", "LA_CALL_COMMIT", "LA_KERNEL_TOKENS",
                       "LA_KERNEL_FEW", "LA_KERNEL_CHUNKED", "LA_KERNEL_CHUNKED_F32")) + "return 0;}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{ROOT}/include", str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(la.LaLaunchInfo), *(getattr(la.LaLaunchInfo, n).offset for n, _ in la.LaLaunchInfo._fields_),
                   0, 1, 2, 3, 0, 1, 2, 3]


def test_timed_prompts():
    short = _info(PREFILL, _shape(8, 160, 16, 48, tokens=700))
    assert (short.kernel, short.state_cols, short.launches) == (CHUNKED, 64, 1)
    full = _info(PREFILL, _shape(8, 2048, 16, 48, tokens=8 * 2048))
    assert (full.kernel, full.state_cols, full.launches, full.workgroups) == (CHUNKED, 128, 1, 8 * 48)
    long = _info(PREFILL, _shape(1, 16384, 16, 32, state=BF16, tokens=16384))
    assert (long.kernel, long.state_cols, long.segment_tokens) == (CHUNKED, 128, 1024)
    odd = _info(PREFILL, _shape(5, 777, 2, 6, 96, 72, x=F32, tokens=1900))
    assert (odd.kernel, odd.segment_tokens, odd.launches) == (CHUNKED_F32, 128, 3)


def test_timed_few_tokens():
    assert _info(UPDATE, _shape(1, 1, 16, 48)).kernel == TOKENS
    full = _info(UPDATE, _shape(256, 1, 32, 32))
    assert (full.kernel, full.streaming, full.launches) == (FEW, 1, 1)
    for call in (VERIFY, COMMIT):
        few = _info(call, _shape(8, 17, 16, 32, state=BF16))
        assert (few.kernel, few.streaming, few.workgroups) == (FEW, 0, 256)
        full = _info(call, _shape(128, 8, 16, 48))
        assert (full.kernel, full.streaming) == (FEW, 1)


@pytest.mark.parametrize("state", [F32, BF16])
def test_tiles_of_prompts(state):
    """128 columns of more than 64 where a launch fills the card, or has chains to fill it with."""
    def cols(n_seq, T, hv, dv=128):
        return _info(PREFILL, _shape(n_seq, T, 1, hv, dv=dv, state=state, tokens=n_seq * T)).state_cols

    assert cols(66, 200, 8) == 128 and cols(64, 200, 8) == 64       # chains of 4 chunks: over 512 workgroups
    assert cols(64, 257, 8) == 128                                  # a chain of 5 chunks
    assert cols(33, 400, 4) == 128 and cols(32, 400, 4) == 64       # over 128 workgroups
    assert cols(66, 200, 8, dv=64) == 64 and cols(66, 200, 8, dv=72) == 128
    assert cols(40, 130, 4) == 64


@pytest.mark.parametrize("hv", [1, 4, 48])
@pytest.mark.parametrize("x", [BF16, F32])
def test_segments_of_prompts(x, hv):
    chunk = 64 if x == BF16 else 32
    for T in (1, chunk, 8 * chunk, 9 * chunk, 4000, 40000):
        info = _info(PREFILL, _shape(1, T, 1, hv, x=x, tokens=T))
        assert info.segment_tokens % chunk == 0
        if T <= 8 * chunk:
            assert info.launches == 1
        if T >= 4000:
            assert info.launches == 3 and info.segment_tokens >= 4 * chunk
    assert _info(PREFILL, _shape(600, 1000, 1, hv, x=x, tokens=600 * 1000)).launches == 1 or hv == 1


@pytest.mark.parametrize("call", [UPDATE, VERIFY, COMMIT])
def test_kernels_of_few_tokens(call):
    one = 16 if call == COMMIT else 12                             # from here on one chunk of fp32 tokens
    for T in (1, 2, 11, one - 1):
        assert _info(call, _shape(3, T, 2, 2, x=F32)).kernel == TOKENS
    for T in (one, 32):
        assert _info(call, _shape(3, T, 2, 2, x=F32)).kernel == CHUNKED_F32
        assert _info(call, _shape(3, T, 2, 2, x=F32, far=1 << 24)).kernel == TOKENS
    for T in (2, 32):
        assert _info(call, _shape(1, T, 1, 1)).kernel == FEW
    assert _info(call, _shape(10, 1, 16, 48)).kernel == TOKENS     # 480 workgroups
    assert _info(call, _shape(11, 1, 16, 48)).kernel == FEW        # 528
    assert _info(call, _shape(32, 2, 16, 48)).streaming == 0       # 96 MiB of states
    assert _info(call, _shape(33, 2, 16, 48)).streaming == 1


def test_prompts_of_tokens_far_apart():
    assert _info(PREFILL, _shape(1, 9, 1, 1, far=(1 << 24) - 8, tokens=9)).kernel == CHUNKED
    assert _info(PREFILL, _shape(1, 9, 1, 1, far=1 << 24, tokens=9)).kernel == TOKENS


def test_refusals_and_nothing_to_do():
    assert _info(PREFILL, _shape(0, 5, 1, 1)).launches == 0
    lib, info = la.load(), la.LaLaunchInfo()
    for call, shape, to in ((4, _shape(1, 1, 1, 1), info), (-1, _shape(1, 1, 1, 1), info),
                            (UPDATE, None, info), (UPDATE, _shape(1, 33, 1, 1), info)):
        assert lib.linattn_describe(call, shape, ctypes.byref(to)) < 0 and lib.linattn_last_error()
    assert lib.linattn_describe(UPDATE, _shape(1, 1, 1, 1), None) == base.CV_EINVAL
