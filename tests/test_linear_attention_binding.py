"""What the binding refuses before it fills the C structures (CPU tensors; the device check and the
launch taken out), and that the call module leaves the same calls to it."""

import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def m(monkeypatch):
    from causal_conv1d_verify_amd import _linattn, linear_attention

    if not os.path.exists(_linattn.LIB_PATH):
        pytest.skip("liblinattn.so not built (run __graft_entry__.build())")
    monkeypatch.setattr(linear_attention, "_same_gpu", lambda first, *others: first.device)
    monkeypatch.setattr(linear_attention, "_on_stream", lambda stream, dev: 0)
    return linear_attention


def _prompt(T=5, device="cpu"):
    q, v = (torch.zeros(T, h, 64, dtype=torch.bfloat16, device=device) for h in (2, 4))
    state = torch.zeros(1, 4, 64, 64, device=device)
    return (q, q, v, None, state, torch.zeros_like(v)), torch.tensor([0, T], dtype=torch.int32, device=device)


@pytest.mark.parametrize("max_len", [2 ** 31, 2 ** 32 + 3, 2 ** 40])
def test_max_len_past_32_bits(m, max_len):
    """Its low 32 bits would be another bound, and rows past that are skipped."""
    args, cu = _prompt()
    with pytest.raises(ValueError, match="max_len"):
        m._attn_args("prefill", *args, cu_seqlens=cu, max_len=max_len)
    m._attn_args("prefill", *args, cu_seqlens=cu, max_len=2 ** 31 - 1)
