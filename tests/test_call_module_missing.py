"""Without the call module (not built, or built for another torch or Python) the binding takes every
call, and says so once."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
torch = pytest.importorskip("torch")

_BLOCKED = """
import sys, warnings
sys.modules["causal_conv1d_verify_amd._lacall"] = None
import torch, causal_conv1d_verify_amd as cv
"""


def _run(code, **env):
    from causal_conv1d_verify_amd import _linattn

    if not os.path.exists(_linattn.LIB_PATH):
        pytest.skip("liblinattn.so not built (run __graft_entry__.build())")
    run = subprocess.run([sys.executable, "-c", _BLOCKED + code], capture_output=True, text=True, cwd=ROOT,
                         env=dict(os.environ, **env), timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    return run.stdout.split()


def test_calls_take_the_binding_and_one_warning():
    assert _run("""
t = torch.zeros(2, 3, 4, 64)
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    for call in (lambda: cv.linear_attn_update(t, t, t, None, torch.zeros(2, 4, 64, 64), t),
                 lambda: cv.gated_norm(t[0], None, torch.zeros(64), t[0]),
                 lambda: cv.residual_norm(t[0, 0], t[0, 0], None, None)):
        try:
            call()
        except ValueError as e:
            print("same" if "same GPU" in str(e) else e)
print(sum(issubclass(w.category, RuntimeWarning) for w in said))
""", HIP_VISIBLE_DEVICES="-1") == ["same", "same", "same", "1"]


@pytest.mark.gpu
def test_calls_run():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("[case] no call module", flush=True)
    assert _run("""
y = torch.randn(5, 2, 64, device="cuda")
out = torch.zeros_like(y)
cv.gated_norm(y, None, torch.ones(64, device="cuda"), out)
torch.cuda.synchronize()
want = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
print((out - want).abs().max().item() < 1e-5)
""") == ["True"]
