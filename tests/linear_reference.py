"""Decayed linear attention and the two norms in 64 bits, from their definitions, with the
bounds that the kernels' results are held to.

Bounds.  A result is off by the rounding of its own type (half a step: eps / 2 of its value)
plus what 32-bit arithmetic inside may lose, which is relative to the same sums taken over
absolute values ("mass").  Inside, a value passes through fewer than dk + T + 128 additions
and products of 32 bits each (the sum over dk, one step for each token, a fixed number more),
and a decay exp(x) carries |x| <= 128 half steps from its argument: (dk + T + 256) * 2^-24 in
all.  Where bf16 tensors go through the matrix cores, 32-bit factors are taken as two bf16
parts, each leaving at most 2^-18 of the factor: three such factors (the state, the decayed
products, the decayed keys or values) make 2^-16.  A 32-bit state takes three parts instead
(2^-24, within the count above).
"""

import math

import torch


def recurrence(q, k, v, g, first, scale, lengths=None):
    """Rows [n, T, heads, channels] (any float type; g [n, T, Hv]) from the states `first`
    [n, Hv, dk, dv]: (out, last, out_mass, last_mass) in 64 bits; rows stop after `lengths`."""
    f = torch.float64
    n, T, hv, dv = v.shape
    group = torch.arange(hv) // (hv // k.shape[2])
    S = first.to(f).clone()
    M = S.abs()
    out = torch.zeros(n, T, hv, dv, dtype=f)
    mass = torch.zeros_like(out)
    for t in range(T):
        on = torch.ones(n, dtype=torch.bool) if lengths is None else torch.as_tensor(lengths) > t
        a = torch.exp(g[:, t].to(f))[..., None, None]
        kt, vt, qt = k[:, t].to(f)[:, group], v[:, t].to(f), q[:, t].to(f)[:, group]
        new = S * a + kt[..., :, None] * vt[..., None, :]
        big = M * a + kt.abs()[..., :, None] * vt.abs()[..., None, :]
        S = torch.where(on[:, None, None, None], new, S)
        M = torch.where(on[:, None, None, None], big, M)
        out[:, t] = scale * (qt[..., None, :] @ new)[..., 0, :]
        mass[:, t] = abs(scale) * (qt.abs()[..., None, :] @ big)[..., 0, :]
    return out, S, mass, M


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def bounds(value, mass, dtype, x_dtype, dk, T):
    """Element by element, how far a result stored as `dtype` may be from `value`."""
    loss = (dk + T + 256) * 2.0 ** -24
    if x_dtype == torch.bfloat16 and not (dtype == torch.float32):
        loss += 2.0 ** -16
    tiny = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
    return half_step(dtype) * value.abs() * (1 + loss) + loss * mass + tiny


def rms(x, weight, eps):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()


def act(z, name):
    z = z.double()
    s = torch.sigmoid(z)
    return s * z if name == "silu" else s


def check(got, value, allowed, what):
    """got within `allowed` of `value` everywhere; reports the worst share of the bound."""
    err = (got.double().cpu() - value).abs()
    assert torch.isfinite(err).all(), f"{what}: not finite"
    share = (err / allowed).max().item() if err.numel() else 0.0
    assert share <= 1.0, f"{what}: {share:.3g} of the bound"
    return share


def spread(count, seed):
    return torch.Generator().manual_seed(seed * 1000003 + count)


def log_decays(shape, gen):
    rate = 1 + 15 * torch.rand(shape[-1], generator=gen)
    return -(rate * torch.nn.functional.softplus(torch.randn(shape, generator=gen) - 3.0))


def scale_of(dk):
    return 1.0 / math.sqrt(dk)
