"""64-bit forms of the selective scan, the rotation of normed heads and the verdict on drafts, with
the bounds that fp32 arithmetic has to keep to.

u = 2^-24 is half a step of fp32.  The bounds are first-order running errors.

Scan.  The kernel's softplus is off by at most 8 u of its value by its own operations and by 2 |v| u
through its argument v = dt + dt_bias (rounded, and scaled for the exponential); its decay
exp(delta A) by the exponent's error, |delta A| (8 + 2 |v| + 3) u, and 2 u; delta x B by that of delta
and 3 u; each update rounds its product and sum (2 u).  With M the recurrence of magnitudes,
M <- a M + delta |x B|, the error E of a state runs as

    E <- a E + a M (|delta A| (11 + 2 |v|) + 4) u + delta |x B| (13 + 2 |v|) u

Where a row is cut the entering state is a sum of such parts, whose decays are of sums of delta: each
sum of n terms is off by n u more at most, which enters as the exponents' errors above do (n is
counted by `L_u`, one more u of |delta A| for each token).  The outputs sum n_states products (n + 2 u
each of them), add D x and are scaled by the gate, which is off by 10 u; then they are rounded to their
type, as the last state is: half a step each.  A state whose M comes to 2^127 may pass fp32's range
(its parts sum to M, whose double fp32 does not hold): from there on it, and what it reaches, may be
anything, and its bound is not finite.
"""

import torch

U = 2.0 ** -24
F64 = torch.float64
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


class Scan:
    """One row, token by token in 64 bits: outputs, states and their bounds."""

    def __init__(self, h, A, D=None, dt_bias=None, use_softplus=True):
        self.h, self.A = h.to(F64).clone(), A.to(F64)
        self.M, self.E = self.h.abs(), torch.zeros_like(self.h)
        self.D = None if D is None else D.to(F64)
        self.bias = None if dt_bias is None else dt_bias.to(F64)
        self.softplus = use_softplus

    def token(self, x, dt, B, C=None, z=None):
        x, v, B = x.to(F64), dt.to(F64), B.to(F64)
        if self.bias is not None:
            v = v + self.bias
        delta = softplus(v) if self.softplus else v
        per = (2 * v.abs() + 11 if self.softplus else torch.full_like(v, 5.0))[:, None]
        arg = delta[:, None] * self.A
        a = torch.exp(arg)
        add = (delta * x)[:, None] * B
        # one more u of each exponent for the token's place in a sum of delta
        self.E = a * self.E + a * self.M * (arg.abs() * (per + 1) + 4) * U + \
            add.abs() * (per + 2) * U
        self.h = a * self.h + add
        self.M = a * self.M + add.abs()
        self.E = torch.where(self.M < 2.0 ** 127, self.E, float("inf"))
        if C is None:
            return None
        C = C.to(F64)
        n = C.shape[0]
        y, bound = self.h @ C, (self.E + (n + 2) * U * self.M) @ C.abs()
        if self.D is not None:
            y, bound = y + self.D * x, bound + 3 * U * (self.D * x).abs()
        if z is not None:
            z = z.to(F64)
            gate = z / (1 + torch.exp(-z))
            y, bound = y * gate, bound * gate.abs() + 10 * U * (y * gate).abs()
        return y, bound + 2 * U * y.abs()

    def state(self):
        return self.h, self.E + 2 * U * self.M


def rounded(value, bound, dtype):
    """The bound with the rounding to dtype: half a step of what is rounded, and half the smallest
    step."""
    return bound + HALF[dtype] * (value.abs() + bound) + (2.0 ** -149 if dtype == torch.float32 else 2.0 ** -134)


def rotary(x, w, positions, inv_freq, eps, interleaved):
    """x [tokens, heads, dim] in 64 bits, and the bound.  The sum of dim squares is off by (16 + 8) u
    (16 in a lane, a few steps across), its root by half of that and 4 u, u w by 3 u more: 19 u.  Sine
    and cosine are off by 4 u: their argument in fp32 (2 u), their series and its roundings (2 u), and
    the products and their sum by 2 u."""
    y = x.to(F64)
    rel = 0.0
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.to(F64)
        rel = 19.0
    out, bound = y.clone(), rel * U * y.abs()
    if inv_freq is not None and len(inv_freq):
        r = len(inv_freq)
        angle = (positions.to(F64)[:, None] * inv_freq.to(F64))[:, None]
        i = torch.arange(r, device=x.device)
        e, f = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        c, s = torch.cos(angle), torch.sin(angle)
        out[..., e] = y[..., e] * c - y[..., f] * s
        out[..., f] = y[..., f] * c + y[..., e] * s
        both = (rel + 6) * U * (y[..., e].abs() + y[..., f].abs())
        bound[..., e] = bound[..., f] = both
    return out, bound


def weights(p, q=None, gone=()):
    w = p.to(F64).clone() if q is None else p.to(F64) - q.to(F64)
    w = torch.where((w > 0) & torch.isfinite(w), w, 0.0)
    for g in gone:
        w[g] = 0
    return w


def verdict(tokens, target, uniform, draft=None, parent=None):
    """One row (lists and CPU tensors): (num_tokens, next_token, window_index, path), or None where
    its parents are not a tree."""
    T, vocab = target.shape
    tokens = [int(t) for t in tokens]
    up = [int(x) for x in parent] if parent is not None else [t - 1 for t in range(T)]
    if up[0] != -1 or any(not -1 <= up[t] < t for t in range(1, T)):
        return None
    u = uniform.to(F64)
    at, way, j = 0, [0], 0
    gone, left, tried = [], 1.0, False
    while True:
        j += 1
        if j >= T:
            break
        if up[j] != at or not 0 <= tokens[j] < vocab:
            continue
        x = tokens[j]
        tried = True
        if x in gone:
            continue
        p = float(target[at, x])
        q = float(draft[at, x]) if draft is not None else left
        if float(u[j - 1]) * q < p:
            at, gone, left, tried = j, [], 1.0, False
            way.append(j)
        else:
            left -= p
            gone.append(x)
    w = weights(target[at], draft[at], ()) if tried and draft is not None else weights(target[at], None, gone)
    if not bool((w > 0).any()):
        w = weights(target[at])
    if not bool((w > 0).any()):
        nxt = -1
    else:
        sums = w.cumsum(0)
        over = (sums > u[T - 1] * sums[-1]).nonzero()
        nxt = int(over[0]) if len(over) else int((w > 0).nonzero()[-1])
    return len(way), nxt, at, way + [-1] * (T - len(way))
