"""GPU tests of the gated head norm and the norm at a block's end against 64 bits.

Bounds.  A result is rounded once to its type (half a step).  Inside, 32-bit steps: the sum of
squares of dim values (its relative error at most (dim / lanes + 16) half steps of 2^-24, and
the root halves it), the quotient and root (2 each), three products, and the gate's
exponential and reciprocal (at most 8 for |z| <= 8, and |z| / ln 2 more for the exponential's argument):
64 + dim / 64 + 2 |z| half steps cover them, relative to the result; the residual sum's error
is relative to the absolute values that it adds.
"""

import math

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
POISON = 7.25


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import causal_conv1d_verify_amd._linattn as L

    L.load()


def _say(*a):
    print("[case]", *a, flush=True)


def _loss(dim, z=None):
    steps = 64 + dim / 64 + (0 if z is None else 2 * z.double().abs())
    return steps * 2.0 ** -24


def _padded(shape, gen, dtype, gap=8, factor=1.0):
    """A tensor with `gap` elements behind each innermost row, on the GPU."""
    full = (factor * torch.randn(*shape[:-1], shape[-1] + gap, generator=gen)).to(dtype).cuda()
    return full[..., :shape[-1]]


def _gated_expected(y, z, w, eps, name, first):
    y, w = y.cpu(), w.cpu()
    if z is None:
        return ref.rms(y, w, eps)
    a = ref.act(z.cpu(), name)
    return ref.rms(y.double() * a, w, eps) if first else ref.rms(y, w, eps) * a


GATED = [(1, 1, 8), (3, 5, 16), (7, 3, 24), (2, 48, 128), (129, 2, 64), (5, 2, 200), (3, 1, 264),
         (2, 3, 512), (4, 1, 1000), (2, 2, 2048), (1000, 4, 128)]


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("name", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gated_norm(shape, dtype, name, first):
    import causal_conv1d_verify_amd as cv

    _say("gated", shape, dtype, name, first)
    gen = ref.spread(shape[2], 3)
    y, z = _padded(shape, gen, dtype), _padded(shape, gen, dtype)
    w = (1 + 0.2 * torch.randn(shape[2], generator=gen)).to(dtype).cuda()
    full = torch.full((*shape[:-1], shape[-1] + 8), POISON, dtype=dtype, device="cuda")
    out = full[..., :shape[-1]]
    cv.gated_norm(y, z, w, out, activation=name, gate_first=first)
    torch.cuda.synchronize()
    want = _gated_expected(y, z, w, 1e-6, name, first)
    loss = _loss(shape[2], z.cpu())
    ref.check(out, want, want.abs() * (ref.half_step(dtype) + loss) + 2.0 ** -126, "out")
    assert (full[..., shape[-1]:] == POISON).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_norm_without_gate_and_in_place(dtype):
    import causal_conv1d_verify_amd as cv

    _say("gated, no gate", dtype)
    gen = ref.spread(1, 4)
    y = _padded((33, 3, 96), gen, dtype)
    w = torch.randn(96, generator=gen).to(dtype).cuda()
    want = _gated_expected(y, None, w, 1e-5, "silu", False)
    cv.gated_norm(y, None, w, y, eps=1e-5)
    torch.cuda.synchronize()
    ref.check(y, want, want.abs() * (ref.half_step(dtype) + _loss(96)) + 2.0 ** -126, "out")
    flat = _padded((9, 96), gen, dtype)
    want = _gated_expected(flat, flat, w, 1e-6, "silu", False)
    out = torch.empty_like(flat)
    cv.gated_norm(flat, flat, w, out)
    torch.cuda.synchronize()
    loss = _loss(96, flat.cpu())
    ref.check(out, want, want.abs() * (ref.half_step(dtype) + loss) + 2.0 ** -126, "2-D")


@pytest.mark.parametrize("dim", [128, 1024])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("power", [-120, -70, 70, 120])
def test_norms_of_extreme_magnitudes(power, eps, dim):
    """Squares outside fp32's range: the sum is taken again over scaled values."""
    import causal_conv1d_verify_amd as cv

    _say("extreme norms", power, eps, dim)
    gen = ref.spread(dim, 6)
    y = torch.ldexp(torch.randn(6, dim, generator=gen), torch.tensor(power)).to(BF16).cuda()
    w = torch.ones(dim, dtype=BF16, device="cuda")
    out = torch.zeros_like(y)
    cv.gated_norm(y, None, w, out, eps=eps)
    want = _gated_expected(y, None, w, eps, "silu", False)
    bound = want.abs() * (ref.half_step(BF16) + _loss(dim)) + 2.0 ** -126
    torch.cuda.synchronize()
    ref.check(out, want, bound, "gated")
    res, nxt = torch.zeros_like(y), torch.zeros_like(y)
    cv.residual_norm(y, res, w, nxt, residual_out=torch.empty_like(res), eps=eps)
    torch.cuda.synchronize()
    ref.check(nxt, want, bound, "residual")


def test_gated_norm_extreme_gates_and_rows_of_zeros():
    import causal_conv1d_verify_amd as cv

    _say("extreme gates")
    z = torch.tensor([-1e30, -200.0, -100.0, -88.0, -80.0, 88.0, 200.0, 1e30], device="cuda")
    y = torch.tensor([[1.0, -2.0, 3.0, 1.0, 1.0, 1.0, 1.0, -1.0], [0.0] * 8], device="cuda")
    w = torch.ones(8, device="cuda")
    for name in ("silu", "sigmoid"):
        out = torch.full_like(y, POISON)
        cv.gated_norm(y, z.expand(2, 8), w, out, activation=name)
        torch.cuda.synchronize()
        want = _gated_expected(y, z, w, 1e-6, name, False)
        assert (out[1] == 0).all()
        # a gate's exponential carries its argument's half steps: 200 of them at most
        ref.check(out, want, want.abs() * 512 * 2.0 ** -24 + 2.0 ** -126, name)


def test_a_row_that_is_not_finite_stays_alone():
    import causal_conv1d_verify_amd as cv

    _say("not finite")
    gen = ref.spread(2, 8)
    for dim in (64, 1024):
        y = torch.randn(6, dim, generator=gen).to(BF16).cuda()
        w = torch.ones(dim, dtype=BF16, device="cuda")
        y[2, 5] = math.nan
        y[4, 1] = math.inf
        want = ref.rms(y.cpu(), w.cpu(), 1e-6)
        rest = [0, 1, 3, 5]
        out, nxt, res = torch.zeros_like(y), torch.zeros_like(y), torch.zeros_like(y)
        cv.gated_norm(y, None, w, out)
        cv.residual_norm(y, res, w, nxt, post_weight=w)
        torch.cuda.synchronize()
        for t in (out, nxt):
            assert torch.isfinite(t[rest]).all() and not torch.isfinite(t[2]).any()
            assert not torch.isfinite(t[4, 1])
        ref.check(out[rest], want[rest], want[rest].abs() * (ref.half_step(BF16) + _loss(dim)), "rest")


RESIDUAL = [(1, 8), (5, 64), (3, 512), (2, 520), (7, 1000), (4, 2048), (3, 4096), (2, 5120),
            (2, 8192), (3, 12296), (2, 16384), (1030, 256)]
TYPES = {"f32": (F32, F32), "bf16": (BF16, BF16), "bf16_f32": (BF16, F32)}


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", RESIDUAL, ids=str)
def test_residual_norm(shape, types, gate, post):
    import causal_conv1d_verify_amd as cv

    _say("residual", shape, types, gate, post)
    xt, rt = TYPES[types]
    gen = ref.spread(shape[1], 7)
    dim = shape[1]
    y, res = _padded(shape, gen, xt), _padded(shape, gen, rt, factor=2.0)
    z = {"none": None, "token": _padded(shape, gen, xt),
         "channel": torch.randn(dim, generator=gen).to(xt).cuda()}[gate]
    pw = (1 + 0.2 * torch.randn(dim, generator=gen)).to(xt).cuda() if post else None
    w = (1 + 0.2 * torch.randn(dim, generator=gen)).to(xt).cuda()
    full = torch.full((shape[0], dim + 8), POISON, dtype=xt, device="cuda")
    res_full = torch.full((shape[0], dim + 8), POISON, dtype=rt, device="cuda")
    kept = res.clone()
    cv.residual_norm(y, res, w, full[:, :dim], post_weight=pw, gate=z, scale=0.7,
                     residual_out=res_full[:, :dim], eps=1e-5)
    torch.cuda.synchronize()
    u = ref.rms(y.cpu(), pw.cpu(), 1e-5) if post else y.cpu().double()
    if z is not None:
        u = u * z.cpu().double()
    scale = float(torch.tensor(0.7))             # as the 32-bit argument holds it
    r = res.cpu().double() + scale * u
    out = ref.rms(r, w.cpu(), 1e-5)
    loss = _loss(dim)
    mass = res.cpu().double().abs() + (scale * u).abs()
    ref.check(res_full[:, :dim], r, r.abs() * ref.half_step(rt) + mass * loss, "residual")
    by = out.abs() / r.abs().clamp(min=1e-30) * mass
    ref.check(full[:, :dim], out, out.abs() * (ref.half_step(xt) + loss) + by * loss + 2.0 ** -126, "out")
    assert (full[:, dim:] == POISON).all() and (res_full[:, dim:] == POISON).all()
    assert torch.equal(res, kept)
    # in place, and without the next norm: the same residual bits
    for args in ((w, torch.empty(shape, dtype=xt, device="cuda")), (None, None)):
        again = kept.clone()
        cv.residual_norm(y, again, *args, post_weight=pw, gate=z, scale=0.7, eps=1e-5)
        torch.cuda.synchronize()
        assert torch.equal(again, res_full[:, :dim])
