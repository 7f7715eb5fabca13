"""The workspace that a prompt's call makes for itself belongs to the stream that the call runs on:
a block that another stream has given up may still be in use by what is queued there."""

import contextlib
import os

import pytest

torch = pytest.importorskip("torch")


def _module():
    from causal_conv1d_verify_amd import _linattn, linear_attention

    if not os.path.exists(_linattn.LIB_PATH):
        pytest.skip("liblinattn.so not built (run __graft_entry__.build())")
    return linear_attention


def _prompt(device, T=3000):
    """Arguments of a prompt that is cut, and so needs a workspace."""
    q, v = (torch.zeros(T, h, 64, dtype=torch.bfloat16, device=device) for h in (1, 2))
    state = torch.zeros(1, 2, 64, 64, device=device)
    cu = torch.tensor([0, T], dtype=torch.int32, device=device)
    return (q, q, v, None, state, torch.empty_like(v)), dict(cu_seqlens=cu, max_len=T)


@pytest.mark.parametrize("handle", [77, 0])
def test_made_under_the_stream_of_the_call(handle, monkeypatch):
    m = _module()
    now = ["current"]
    made = []

    @contextlib.contextmanager
    def under(stream):
        now.append(stream)
        yield
        now.pop()

    class Current:
        cuda_stream = 5

    empty = torch.empty
    monkeypatch.setattr(m, "_same_gpu", lambda first, *others: first.device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: h)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(now[-1]) or empty(*a, **kw))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    args, kw = _prompt("cpu")
    made.clear()
    keep = m._attn_args("prefill", *args, **kw, stream=handle)[-1]
    assert keep[-1].numel() > 0 and made == [handle]
    made.clear()
    m._attn_args("prefill", *args, **kw, stream=Current)
    assert made == ["current"]


@pytest.mark.gpu
@pytest.mark.parametrize("way", ["other", "default"])
def test_block_of_the_stream_of_the_call(way):
    """No launch: where the block comes from, beside one of the same size that the current stream
    has just given up."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("[case] workspace", way, flush=True)
    m = _module()
    a, b = torch.cuda.Stream(), torch.cuda.default_stream()
    launch, current = (a, b) if way == "other" else (b, a)
    args, kw = _prompt("cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        size = m._attn_args("prefill", *args, **kw)[-1][-1].numel()
        given_up = torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr()
        keep = m._attn_args("prefill", *args, **kw, stream=launch)[-1]
    assert keep[-1].numel() == size and keep[-1].data_ptr() != given_up
    of = [s["stream"] for s in torch.cuda.memory_snapshot()
          if 0 <= keep[-1].data_ptr() - s["address"] < s["total_size"]]
    assert of == [launch.cuda_stream]


@pytest.mark.gpu
def test_beside_work_of_the_current_stream():
    """What is queued on the current stream keeps the block that it gave up while the prompt runs on
    another."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("[case] workspace beside other work", flush=True)
    import causal_conv1d_verify_amd as cv

    m = _module()
    gen = torch.Generator().manual_seed(3)
    (q, _, v, _, state, out), kw = _prompt("cuda")
    k = torch.randn(q.shape, generator=gen).to(q.dtype).cuda()
    v.copy_(torch.randn(v.shape, generator=gen))
    max_len, cu = kw["max_len"], kw["cu_seqlens"]
    cv.linear_attn_prefill(k, k, v, None, state, out, cu, max_len=max_len)
    torch.cuda.synchronize()
    want = out.clone(), state.clone()
    size = m._attn_args("prefill", k, k, v, None, state, out, **kw)[-1][-1].numel()
    a, s = torch.randn(4096, 4096, device="cuda"), torch.cuda.Stream()
    for _ in range(3):
        state.zero_()
        out.zero_()
        s.wait_stream(torch.cuda.current_stream())
        b = a @ a                                  # some milliseconds of work in front
        block = torch.full((size,), 9, dtype=torch.uint8, device="cuda")
        kept = block + 0
        del block
        cv.linear_attn_prefill(k, k, v, None, state, out, cu, max_len=max_len, stream=s)
        torch.cuda.synchronize()
        assert (kept == 9).all() and b.shape == a.shape
        assert torch.equal(out, want[0]) and torch.equal(state, want[1])
