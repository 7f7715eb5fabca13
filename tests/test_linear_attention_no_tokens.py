"""Packed prompts without a single token, under any bound on their length: states are kept, or start
from zeros, and nothing else is asked for."""

import os

import pytest

torch = pytest.importorskip("torch")


def _module():
    from causal_conv1d_verify_amd import _linattn, linear_attention

    if not os.path.exists(_linattn.LIB_PATH):
        pytest.skip("liblinattn.so not built (run __graft_entry__.build())")
    return linear_attention


def _none(device, dtype=torch.bfloat16, rows=3):
    q, v = (torch.empty(0, h, 64, dtype=dtype, device=device) for h in (2, 4))
    state = torch.ones(rows, 4, 64, 64, device=device)
    cu = torch.zeros(rows + 1, dtype=torch.int32, device=device)
    return q, q.clone(), v, torch.empty(0, 4, device=device), state, torch.empty_like(v), cu


@pytest.mark.parametrize("max_len", [0, 1, 2, 64, 100000])
def test_are_taken_without_a_workspace(max_len, monkeypatch):
    m = _module()
    monkeypatch.setattr(m, "_same_gpu", lambda first, *others: first.device)
    monkeypatch.setattr(m, "_on_stream", lambda stream, dev: 0)
    *args, cu = _none("cpu")
    lib, _, _, cargs, keep = m._attn_args("prefill", *args, cu_seqlens=cu, max_len=max_len)
    assert lib.linattn_prefill_workspace(cargs[0]) == 0 and keep[-1] is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("max_len", [1, 2, 64, 100000])
def test_states_are_kept_or_emptied(max_len, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("[case] no tokens", max_len, dtype, flush=True)
    import causal_conv1d_verify_amd as cv

    for started in (None, [1, 0, 1]):
        *args, cu = _none("cuda", dtype)
        init = None if started is None else torch.tensor(started, dtype=torch.int32, device="cuda")
        cv.linear_attn_prefill(*args, cu, max_len=max_len, has_initial_state=init)
        torch.cuda.synchronize()
        for i, keep in enumerate(started or [1, 1, 1]):
            assert (args[4][i] == keep).all()
