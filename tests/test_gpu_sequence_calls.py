"""The call module of libseqops.so takes the calls that are plainly in order, and both ways give the same
bits; other devices, streams and shapes go the binding's way."""

import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


def _need():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import causal_conv1d_verify_amd as cv

    return cv


def _calls():
    """name -> (arguments of the call module, the entry point on a stream, what it writes), on fresh buffers."""
    cv = _need()
    gen = torch.Generator().manual_seed(3)

    def n(*shape, dtype=BF16):
        return torch.randn(*shape, generator=gen).to(dtype).cuda()

    x, dt, z, low = n(3, 4, 88)[..., :72], n(3, 4, 72), n(3, 4, 72), n(3, 4, 35)
    B, C = low[..., 1:17], low[..., 17:33]
    A, D, bias = -n(72, 16, dtype=torch.float32).abs(), n(72, dtype=torch.float32), n(72, dtype=torch.float32)
    pool = n(5, 72, 16, dtype=torch.float32)
    slots = torch.tensor([4, -1, 2], dtype=torch.int32).cuda()
    num = torch.tensor([2, 1, 4], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 5, 5, 12], dtype=torch.int32).cuda()
    init = torch.tensor([1, 0, 0], dtype=torch.int32).cuda()
    calls = {}

    def scan(kind, name):
        S, out = pool.clone(), torch.zeros(3, 4, 72, dtype=BF16, device="cuda")
        flat = (lambda t: t.flatten(0, 1)) if kind == 0 else (lambda t: t)
        xs, dts, zs, Bs, Cs, o = (flat(t) for t in (x, dt, z, B, C, out))
        if kind == 3:
            args = (3, xs, dts, A, Bs, None, S, None, None, None, None, None, bias, True, slots, None, num, None)
            call = lambda stream: cv.selective_scan_commit(xs, dts, A, Bs, S, num, dt_bias=bias, slot_idx=slots, stream=stream)
        else:
            kw = dict(z=zs, D=D, dt_bias=bias, slot_idx=slots)
            more = (cu,) if kind == 0 else ()
            if kind == 0:
                kw.update(max_len=7, has_initial_state=init)
            args = (kind, xs, dts, A, Bs, Cs, S, o, cu if kind == 0 else None, 7 if kind == 0 else None, zs, D, bias, True, slots,
                    init if kind == 0 else None, None, None)
            call = lambda stream: getattr(cv, name)(xs, dts, A, Bs, Cs, S, o, *more, stream=stream, **kw)
        return "scan", args, call, (S, out)

    for kind, name in enumerate(("prefill", "update", "verify", "commit")):
        calls["selective_scan_" + name] = lambda kind=kind, name=name: scan(kind, "selective_scan_" + name)

    def rotary():
        q, k = n(6, 3, 80)[..., :64], n(6, 2, 64)
        pos, freq = torch.arange(6).cuda() + 100, torch.rand(16, generator=gen).cuda()
        outs = torch.zeros(6, 3, 64, dtype=BF16, device="cuda"), torch.zeros(6, 2, 64, dtype=BF16, device="cuda")
        w = n(64)
        return ("rotary", (q, k, pos, freq, *outs, w, w, 1e-5, True),
                lambda stream: cv.qk_norm_rotary(q, k, pos, freq, *outs, q_weight=w, k_weight=w, eps=1e-5, interleaved=True, stream=stream),
                outs)

    def accept():
        p, d = n(4, 3, 501, dtype=torch.float32).softmax(-1)[..., :500], n(4, 2, 500, dtype=torch.float32).softmax(-1)
        t, u = torch.randint(0, 500, (4, 3), generator=gen).int().cuda(), torch.rand(4, 3, generator=gen).cuda()
        outs = [torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(3)] + [torch.zeros(4, 3, dtype=torch.int32, device="cuda")]
        s = torch.tensor([0, -1, 5, 2], dtype=torch.int32).cuda()
        return ("accept", (t, p, u, outs[0], outs[1], d, None, outs[2], outs[3], s, None),
                lambda stream: cv.accept_drafts(t, p, u, outs[0], outs[1], draft=d, window_index=outs[2], path=outs[3], slot_idx=s,
                                                stream=stream), outs)

    calls["qk_norm_rotary"], calls["accept_drafts"] = rotary, accept
    return calls


NAMES = ["selective_scan_prefill", "selective_scan_update", "selective_scan_verify", "selective_scan_commit",
         "qk_norm_rotary", "accept_drafts"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_taken_and_the_same_bits(name):
    _need()
    from causal_conv1d_verify_amd import _sqcall

    print("[case]", name, flush=True)
    torch.cuda.set_device(0)
    fn, args, _, short = _calls()[name]()
    assert getattr(_sqcall, fn)(*args) == 0
    _, _, call, plain = _calls()[name]()
    call(None)
    _, _, call, named = _calls()[name]()
    call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for a, b, c in zip(short, plain, named):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert any(bool((t != 0).any()) for t in short)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_refusals_of_the_library_are_raised(name):
    """An argument that only the library refuses: the same error on both ways, and nothing written."""
    cv = _need()
    print("[case]", name, flush=True)
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    x, B, A, S = z(2, 3, 60), z(2, 3, 16), z(60, 16, dtype=torch.float32), z(2, 60, 16, dtype=torch.float32)
    calls = {"selective_scan_prefill": lambda s: cv.selective_scan_prefill(x[0], x[0], A, B[0], B[0], S, x[0].clone(), i, max_len=3, stream=s),
             "selective_scan_update": lambda s: cv.selective_scan_update(x, x, A, B, B, S, x.clone(), stream=s),
             "selective_scan_verify": lambda s: cv.selective_scan_verify(x, x, A, B, B, S, x.clone(), stream=s),
             "selective_scan_commit": lambda s: cv.selective_scan_commit(x, x, A, B, S, stream=s),
             "qk_norm_rotary": lambda s: cv.qk_norm_rotary(z(2, 3, 24), None, None, None, z(2, 3, 24), None, stream=s),
             "accept_drafts": lambda s: cv.accept_drafts(z(2, 33, dtype=torch.int32), z(2, 33, 9), z(2, 33, dtype=torch.float32), i, i, stream=s)}
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(cv.SeqOpsError, match="not supported"):
            calls[name](stream)


_BLOCKED = """
import sys, warnings
sys.modules["causal_conv1d_verify_amd._sqcall"] = None
import torch, causal_conv1d_verify_amd as cv
"""


def _run(code, **env):
    from causal_conv1d_verify_amd import _seqops

    if not os.path.exists(_seqops.LIB_PATH):
        pytest.skip("libseqops.so not built (run __graft_entry__.build())")
    run = subprocess.run([sys.executable, "-c", _BLOCKED + code], capture_output=True, text=True, cwd=ROOT,
                         env=dict(os.environ, **env), timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    return run.stdout.split()


def test_without_the_call_module_the_binding_and_one_warning():
    assert _run("""
x, B, A, S = torch.zeros(2, 3, 64), torch.zeros(2, 3, 16), torch.zeros(64, 16), torch.zeros(2, 64, 16)
i = torch.zeros(2, 1, dtype=torch.int32)
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    for call in (lambda: cv.selective_scan_update(x, x, A, B, B, S, x), lambda: cv.selective_scan_commit(x, x, A, B, S),
                 lambda: cv.qk_norm_rotary(x, None, None, None, x, None),
                 lambda: cv.accept_drafts(i, x[:, :1], torch.zeros(2, 1), i[:, 0], i[:, 0])):
        try:
            call()
        except ValueError as e:
            print("same" if "same GPU" in str(e) else e)
print(sum(issubclass(w.category, RuntimeWarning) for w in said))
""", HIP_VISIBLE_DEVICES="-1") == ["same"] * 4 + ["1"]


@pytest.mark.gpu
def test_calls_run_without_the_call_module():
    _need()
    print("[case] no call module", flush=True)
    assert _run("""
q = torch.randn(5, 2, 64, device="cuda")
out = torch.zeros_like(q)
cv.qk_norm_rotary(q, None, None, None, out, None, q_weight=torch.ones(64, device="cuda"))
torch.cuda.synchronize()
want = q / (q.square().mean(-1, keepdim=True) + 1e-6).sqrt()
print((out - want).abs().max().item() < 1e-5)
""") == ["True"]
