"""GPU tests of the norm of q and k heads with their rotation, against the 64-bit form and bounds of
sequence_reference.py."""

import pytest
import torch

import sequence_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
POISON = 7.25


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from causal_conv1d_verify_amd import _seqops

    _seqops.load()


def _cv():
    import causal_conv1d_verify_amd as cv

    return cv


def _say(*a):
    print("[case]", *a, flush=True)


class Problem:
    """q and k as views of one wider buffer, outs with gaps, all around them poison."""

    def __init__(self, tokens, hq, hk, dim, rot, dtype, *, norm=(True, True), first=0, wide=True, seed=1):
        gen = torch.Generator().manual_seed(seed)
        cols = (hq + hk) * dim + 16
        self.rows = torch.randn(tokens, cols, generator=gen).to(dtype).cuda()
        self.q = self.rows[:, :hq * dim].unflatten(1, (hq, dim))
        self.k = self.rows[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim)) if hk else None
        self.w = [(1 + 0.2 * torch.randn(dim, generator=gen)).to(dtype).cuda() if n else None for n in norm]
        if not hk:
            self.w[1] = None
        self.positions = (first + torch.randperm(tokens, generator=gen)).to(torch.int64 if wide else torch.int32).cuda()
        self.inv_freq = (10000.0 ** (-torch.arange(0, rot, 2).float() / max(rot, 1))).cuda() if rot else None
        if not rot:
            self.positions = None
        self.full = [torch.full((tokens, h, dim + 16), POISON, dtype=dtype, device="cuda") if h else None
                     for h in (hq, hk)]
        self.out = [None if t is None else t[..., :dim] for t in self.full]

    def call(self, out=None, **kw):
        out = self.out if out is None else out
        _cv().qk_norm_rotary(self.q, self.k, self.positions, self.inv_freq, *out, q_weight=self.w[0],
                             k_weight=self.w[1], **kw)

    def expect(self, interleaved=False, eps=1e-6):
        res = []
        for x, w in ((self.q, self.w[0]), (self.k, self.w[1])):
            if x is not None:
                r, bound = ref.rotary(x, w, self.positions, self.inv_freq, eps, interleaved)
                res.append((r, ref.rounded(r, bound, x.dtype)))
        return res

    def check(self, want, out=None):
        torch.cuda.synchronize()
        for got, (r, tol) in zip(self.out if out is None else out, want):
            off = (got.double() - r).abs()
            bad = ~(off <= tol)
            assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), off[bad][:4].tolist(),
                                   tol[bad][:4].tolist())
        for full in self.full:
            if full is not None and out is None:
                assert bool((full[..., -16:] == POISON).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(16, 16), (32, 16), (48, 48), (64, 32), (96, 96), (128, 128), (128, 64), (160, 48),
                                     (256, 256), (240, 16), (128, 0)])
@pytest.mark.parametrize("tokens,hq,hk", [(1, 16, 16), (3, 5, 1), (70, 40, 8)])
def test_heads(dtype, interleaved, dim, rot, tokens, hq, hk):
    _say(dtype, interleaved, dim, rot, tokens, hq, hk)
    p = Problem(tokens, hq, hk, dim, rot, dtype, first=1000, seed=dim + rot)
    want = p.expect(interleaved)
    p.call(interleaved=interleaved)
    p.check(want)


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
def test_without_a_norm(norm):
    _say(norm)
    p = Problem(33, 6, 3, 64, 64, F32, norm=norm)
    want = p.expect()
    p.call()
    p.check(want)


def test_q_alone_and_many_tokens():
    _say("q alone")
    p = Problem(5000, 3, 0, 64, 32, BF16)
    want = p.expect()
    p.call()
    p.check(want)


@pytest.mark.parametrize("first,wide", [(2 ** 31 - 70, False), (2 ** 24 + 1, True), (10 ** 7, True), (2 ** 31 + 5, True),
                                        (-64, True), (-2 ** 31, False)])
def test_far_positions(first, wide):
    """The angle is a product in 64 bits, as in the reference, and its remainder modulo a turn is exact
    but for 2^-53 of a turn: what fp32 makes of it does not grow with the position."""
    _say(first, wide)
    p = Problem(64, 2, 2, 64, 64, F32, first=first, wide=wide)
    want = p.expect()
    p.call()
    p.check(want)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_in_place(dtype):
    _say("in place", dtype)
    p = Problem(19, 7, 5, 128, 64, dtype)
    want, gap = p.expect(), p.rows[:, -16:].clone()
    p.call(out=(p.q, p.k))
    p.check(want, out=(p.q, p.k))
    assert torch.equal(p.rows[:, -16:], gap)


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e30])
def test_magnitudes(scale):
    """Sums of squares beyond fp32's range."""
    _say(scale)
    p = Problem(9, 3, 2, 64, 64, F32)
    p.rows.mul_(scale)
    want = p.expect(eps=0.0)
    p.call(eps=0.0)
    p.check(want)


def test_a_head_that_is_not_finite_stays_alone():
    _say("not finite")
    a, b = (Problem(9, 6, 3, 64, 64, BF16) for _ in range(2))
    a.call()
    b.q[4, 2, 7] = float("nan")
    b.k[2, 1, 3] = float("inf")
    b.call()
    torch.cuda.synchronize()
    same = [torch.ones_like(t, dtype=torch.bool) for t in a.out]
    same[0][4, 2] = same[1][2, 1] = False
    for x, y, s in zip(a.out, b.out, same):
        assert torch.equal(x[s], y[s])
    assert torch.isnan(b.out[0][4, 2].float()).all()


def test_a_captured_call_and_a_named_stream():
    _say("graph")
    p = Problem(40, 16, 4, 128, 128, BF16, first=77)
    want = p.expect()
    p.call(stream=torch.cuda.current_stream())
    p.check(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call()
    for _ in range(3):
        for t in p.out:
            t.fill_(POISON)
        graph.replay()
        p.check(want)


def test_no_tokens():
    _say("no tokens")
    p = Problem(0, 2, 2, 64, 64, BF16)
    p.call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("scale", [1e-38, 1e-40, 1e-44])
def test_subnormal_heads(scale):
    """Values that fp32 holds as subnormals (exactly, as the inputs' own), whose norm is an ordinary one."""
    _say(scale)
    p = Problem(9, 3, 2, 64, 32, F32)
    p.rows.mul_(scale)
    want = p.expect(eps=0.0)
    p.call(eps=0.0)
    p.check(want)
