"""The call module: what it takes gives what the binding's own way gives, and what is not plainly
in order is left to that way (None), which says what is wrong."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
torch = pytest.importorskip("torch")


def _module():
    import causal_conv1d_verify_amd._linattn as L

    if not os.path.exists(os.path.join(os.path.dirname(L.LIB_PATH), "_lacall.so")):
        pytest.skip("_lacall.so not built (run __graft_entry__.build())")
    from causal_conv1d_verify_amd import _lacall

    return _lacall


def test_other_arguments_are_left_alone():
    """CPU tensors, no tensors, wrong counts: None, and no exception of the module's own."""
    m = _module()
    t, s = torch.zeros(2, 3, 4, 64), torch.zeros(2, 4, 64, 64)
    i32 = torch.zeros(3, dtype=torch.int32)
    for kind in (0, 1, 2, 3, 7):
        assert m.attn(kind, t, t, t, None, s, t, None, None, None, None, None, None, None) is None
    assert m.attn(0, t[0], t[0], t[0], None, s, t[0], i32, 3, None, None, None, None, None) is None
    assert m.attn(1, None, t, t, None, s, t, None, None, None, None, None, None, None) is None
    assert m.attn(1, "q", 3, t, None, s, t, None, None, None, None, None, None, None) is None
    assert m.attn(1, t) is None and m.attn() is None
    w = torch.zeros(64)
    assert m.gated(t[0], t[0], w, t[0], 1e-6, 0, False) is None
    assert m.gated(t[0], None, w, "out", "eps", 0, False) is None
    assert m.gated(t) is None
    assert m.residual(t[0, 0], t[0, 0], w, t[0, 0], None, None, 1.0, None, 1e-6) is None
    assert m.residual(t[0, 0], None, w, None, None, None, 1.0, None, 1e-6) is None
    assert m.residual() is None


def test_import_needs_no_gpu():
    run = subprocess.run([sys.executable, "-c", "import torch, causal_conv1d_verify_amd as cv\n"
                          "from causal_conv1d_verify_amd import linear_attention as m\n"
                          "print(bool(m._short().attn))"], capture_output=True, text=True, cwd=ROOT,
                         env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"), timeout=300)
    _module()
    assert run.stdout.strip() == "True", run.stderr[-2000:]


def _calls(device="cuda"):
    """name -> (function of (stream) that runs the call on fresh buffers, what it wrote)"""
    import causal_conv1d_verify_amd as cv

    gen = torch.Generator().manual_seed(5)

    def n(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen).to(dtype).to(device)

    q, k, v = n(3, 4, 2, 64), n(3, 4, 2, 64), n(3, 4, 6, 96)[..., :72]
    g = -n(3, 4, 6, dtype=torch.float32).abs()
    pool = n(5, 6, 64, 72, dtype=torch.float32)
    slots = torch.tensor([4, -1, 2], dtype=torch.int32, device=device)
    num = torch.tensor([2, 1, 4], dtype=torch.int32, device=device)
    cu = torch.tensor([0, 5, 5, 12], dtype=torch.int32, device=device)
    init = torch.tensor([1, 0, 0], dtype=torch.int32, device=device)
    y, z, w = n(7, 3, 40), n(7, 3, 48)[..., :40], n(40)
    r, res, wr = n(7, 264)[:, :256], n(7, 256, dtype=torch.float32), n(256)

    def attn(name, *extra, packed=False, outputs=True, **kw):
        def call(stream):
            S, out = pool.clone(), torch.zeros(3, 4, 6, 72, dtype=torch.bfloat16, device=device)
            a = [q, k, v, g, S] if outputs else [k, v, g, S]
            if packed:
                a = [t.flatten(0, 1) if t is not S else t for t in a]
                out = out.flatten(0, 1)
            getattr(cv, name)(*a, *([out] if outputs else []), *extra, slot_idx=slots, stream=stream, **kw)
            return S, out
        return call

    def gated(stream):
        out = torch.zeros_like(y)
        cv.gated_norm(y, z, w, out, activation="sigmoid", gate_first=True, eps=1e-5, stream=stream)
        return (out,)

    def residual(stream):
        out, new = torch.zeros(7, 256, dtype=torch.bfloat16, device=device), res.clone()
        cv.residual_norm(r, new, wr, out, post_weight=wr, gate=wr, scale=0.5, stream=stream)
        return out, new

    return {"prefill": attn("linear_attn_prefill", cu, packed=True, max_len=7, has_initial_state=init),
            "update": attn("linear_attn_update", scale=0.3),
            "verify": attn("linear_attn_verify", scale=2),
            "commit": attn("linear_attn_commit", num, outputs=False),
            "gated": gated, "residual": residual}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["prefill", "update", "verify", "commit", "gated", "residual"])
def test_both_ways_agree(name, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from causal_conv1d_verify_amd import linear_attention as m

    print("[case] both ways", name, flush=True)
    taken = []
    short, done = m._short(), m._done
    monkeypatch.setattr(m, "_done", lambda rc: taken.append(rc) or done(rc))
    call = _calls()[name]
    first = call(None)
    assert taken == [0], "the call module did not take the call"
    second = call(torch.cuda.current_stream())
    assert taken == [0] and short is m._short()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    assert any(t.any() for t in first)


@pytest.mark.gpu
def test_refusals_are_the_same():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import causal_conv1d_verify_amd as cv

    t = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(2, 4, 64, 64, device="cuda")
    stream = torch.cuda.current_stream()
    odd = torch.zeros(2, 3, 4, 60, dtype=torch.bfloat16, device="cuda")
    many = torch.zeros(1, 33, 4, 64, dtype=torch.bfloat16, device="cuda")
    for args, kind in (((odd, odd, t, None, s[:, :, :60].contiguous(), t.clone()), cv.LinAttnError),
                       ((many, many, many, None, s, many.clone()), cv.LinAttnError),
                       ((t, t, t, None, s[:1], t.clone()), cv.LinAttnError),
                       ((t, t, t, None, s.half(), t.clone()), TypeError),
                       ((t, t, t.float(), None, s, t.clone()), TypeError),
                       ((t, t, t, None, s.transpose(2, 3), t.clone()), ValueError),
                       ((t, t, t, None, s.cpu(), t.clone()), ValueError),
                       ((t, t, t, torch.zeros(3, 4, device="cuda"), s, t.clone()), ValueError)):
        said = []
        for kw in ({}, {"stream": stream}):
            with pytest.raises(kind) as e:
                cv.linear_attn_update(*args, **kw)
            said.append(str(e.value))
        assert said[0] == said[1]
