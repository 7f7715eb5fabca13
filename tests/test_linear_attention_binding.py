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


def test_describe_makes_no_workspace(m, monkeypatch):
    args, cu = _prompt(3000)
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(a) or empty(*a, **kw))
    for call in (lambda: m.linear_attn_describe("prefill", *args, cu, max_len=3000),
                 lambda: m.linear_attn_describe("prefill", *args, cu_seqlens=cu, max_len=3000)):
        info = call()
        assert info.launches == 3 and info.workspace_bytes > 0 and not made
    few = [t if t is None or t.dim() > 3 else t[None, :5] for t in args]
    assert m.linear_attn_describe("update", *few).launches == 1
    assert m.linear_attn_describe("commit", *few[1:5]).launches == 1
    with pytest.raises(KeyError):
        m.linear_attn_describe("forward", *few)


def _spread(size, device="cpu"):
    """Tensors of `size` bytes by their count, over fewer or over others' between them."""
    byte = torch.zeros(1, dtype=torch.uint8, device=device)
    return byte.expand(size), torch.zeros(2 * size, dtype=torch.uint8, device=device)[::2]


def test_workspace_that_is_not_whole(m):
    """Its bytes are not where its size says: the kernels would write past or between them."""
    args, cu = _prompt(3000)
    lib, _, _, cargs, _ = m._attn_args("prefill", *args, cu_seqlens=cu, max_len=3000,
                                       workspace=torch.zeros(1, dtype=torch.uint8))
    size = lib.linattn_prefill_workspace(cargs[0])
    assert size > 0
    for workspace in _spread(size):
        with pytest.raises(ValueError, match="workspace"):
            m._attn_args("prefill", *args, cu_seqlens=cu, max_len=3000, workspace=workspace)
    m._attn_args("prefill", *args, cu_seqlens=cu, max_len=3000, workspace=torch.zeros(size, dtype=torch.uint8))


@pytest.mark.gpu
def test_workspace_that_is_not_whole_both_ways():
    """Neither way launches anything with it."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import causal_conv1d_verify_amd as cv

    print("[case] workspace that is not whole", flush=True)
    args, cu = _prompt(3000, "cuda")
    for stream in (None, torch.cuda.current_stream()):
        for workspace in _spread(1 << 26, "cuda"):
            with pytest.raises(ValueError, match="workspace"):
                cv.linear_attn_prefill(*args, cu, max_len=3000, workspace=workspace, stream=stream)
        whole = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
        cv.linear_attn_prefill(*args, cu, max_len=3000, workspace=whole, stream=stream)
        torch.cuda.synchronize()
