"""Random problems of linear attention over the whole argument space, against the recurrence in 64
bits: head counts and sizes, types, lengths, bounds on them, slots and padded rows, first states,
decays of every form and strength, scales, layouts (one buffer of rows, heads before tokens, one key
for all heads, wide gaps), pointers that are 16 but not 32 bytes aligned.  Bounds are those of
linear_reference.py; what a call must not write keeps its bits.
"""

import math
import random

import pytest
import torch

import linear_reference as ref
from test_gpu_linear_attention import BF16, F32, PAIRS, _need_gpu, _say  # noqa: F401

pytestmark = pytest.mark.gpu

POISON = 7.25


def _tokens(rng, gen, shape, dtype, layout):
    """A [..., tokens, heads, channels] tensor of normal values in a layout of its own."""
    *lead, heads, ch = shape
    gap = 8 * rng.randint(0, 3)
    if layout == "heads":                        # heads before tokens
        full = torch.randn(heads, *lead, ch + gap, generator=gen).to(dtype).cuda()
        return full[..., :ch].movedim(0, len(lead))
    full = torch.randn(*lead, heads * ch + 8 + gap, generator=gen).to(dtype).cuda()
    return full[..., 8:8 + heads * ch].unflatten(-1, (heads, ch))


def _poisoned(rng, shape, dtype, layout):
    *lead, heads, ch = shape
    gap = 8 * rng.randint(0, 2)
    if layout == "heads":
        full = torch.full((heads, *lead, ch + gap), POISON, dtype=dtype, device="cuda")
        return full, full[..., :ch].movedim(0, len(lead))
    full = torch.full((*lead, heads, ch + gap), POISON, dtype=dtype, device="cuda")
    return full, full[..., :ch]


def _decays(rng, gen, lead, hv):
    kind = rng.choice(["token", "token", "token", "head", "none", "strong"])
    if kind == "none":
        return None
    if kind == "head":
        return (0.1 * ref.log_decays((1, hv), gen)[0]).cuda()
    g = ref.log_decays((*lead, hv + 3), gen)
    if kind == "strong":
        pick = torch.rand(g.shape, generator=gen)
        g = torch.where(pick < 0.05, -math.inf, torch.where(pick < 0.1, -1000.0, torch.where(pick < 0.3, 0.0, g)))
    return g.cuda()[..., :hv]


def _pool(rng, gen, n, hv, dk, dv, dtype):
    area, gap = hv * dk * dv, 8 * rng.randint(0, 2)
    slots = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32)
    for i in range(n):
        if rng.random() < 0.08:
            slots[i] = rng.choice([-1, -7, n + 2])
    full = torch.randn(n + 2, area + gap, generator=gen).to(dtype).cuda()
    return slots, full, full[:, :area].unflatten(1, (hv, dk, dv))


def _sizes(rng):
    hq = rng.choice([1, 1, 2, 3, 5])
    hv = hq * rng.choice([1, 1, 2, 3, 4])
    dk, dv = (rng.choice([8 * rng.randint(1, 32), 64, 128, 128]) for _ in range(2))
    return hq, hv, dk, dv, rng.choice(list(PAIRS))


def _run(rng, gen, packed):
    import causal_conv1d_verify_amd as cv

    hq, hv, dk, dv, pair = _sizes(rng)
    xt, st = PAIRS[pair]
    if packed:
        n = rng.randint(1, 7)
        top = int(round(math.exp(rng.uniform(0, math.log(1500 if hv * dk * dv < 60000 else 300)))))
        lengths = [rng.randint(0, top) for _ in range(n)]
        lengths[rng.randrange(n)] = top
        T, lead = top, (sum(lengths),)
    else:
        n, T = rng.choice([1, 2, 3, 8, 40]), rng.randint(1, 32)
        lengths, lead = [T] * n, (n, T)
    layouts = [rng.choice(["rows", "rows", "heads"]) for _ in range(4)]
    q, k = (_tokens(rng, gen, (*lead, hq, dk), xt, x) for x in layouts[:2])
    if rng.random() < 0.15:
        k = _tokens(rng, gen, (*lead, 1, dk), xt, "rows").expand(*lead, hq, dk)
    v = _tokens(rng, gen, (*lead, hv, dv), xt, layouts[2])
    full, out = _poisoned(rng, (*lead, hv, dv), xt, layouts[3])
    g = _decays(rng, gen, lead, hv)
    slots, pool_full, pool = _pool(rng, gen, n, hv, dk, dv, st)
    before = pool_full.clone()
    scale = rng.choice([None, None, 1.0, -0.37])
    live = [i for i in range(n) if 0 <= slots[i] < n + 2]
    started = [rng.randint(0, 1) for _ in range(n)] if packed and rng.random() < 0.6 else None
    what = "prefill" if packed else rng.choice(["update", "verify", "commit"])
    counts = lengths if what != "commit" or rng.random() < 0.3 else [rng.randint(0, T) for _ in range(n)]

    with torch.device("cuda"):
        def rows(t):
            if not packed:
                return t
            padded = torch.zeros(n, T, *t.shape[1:], dtype=t.dtype)
            at = 0
            for i, length in enumerate(lengths):
                padded[i, :length] = t[at:at + length]
                at += length
            return padded

        ge = torch.zeros(*lead, hv) if g is None else g.expand(*lead, hv)
        first = torch.zeros(n, hv, dk, dv, dtype=st)
        for i in live:
            if started is None or started[i]:
                first[i] = pool[int(slots[i])]
        want, last, want_mass, last_mass = ref.recurrence(
            rows(q), rows(k), rows(v), rows(ge), first, ref.scale_of(dk) if scale is None else scale,
            torch.tensor(counts))
    i32 = slots.cuda()
    if what == "prefill":
        cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        init = None if started is None else torch.tensor(started, dtype=torch.int32, device="cuda")
        cv.linear_attn_prefill(q, k, v, g, pool, out, cu, max_len=rng.choice([T, T, 2 * T + 5]), scale=scale,
                               slot_idx=i32, has_initial_state=init)
    elif what == "commit":
        cv.linear_attn_commit(k, v, g, pool, None if counts is lengths else
                              torch.tensor(counts, dtype=torch.int32, device="cuda"), slot_idx=i32)
    else:
        getattr(cv, "linear_attn_" + what)(q, k, v, g, pool, out, scale=scale, slot_idx=i32)
    torch.cuda.synchronize()

    worst = [0.0, 0.0]
    got, untouched = out.clone(), full.clone()
    at = 0
    view = untouched[..., :dv].movedim(0, len(lead)) if layouts[3] == "heads" else untouched[..., :dv]
    for i, length in enumerate(lengths):
        mine = got[at:at + length] if packed else got[i]
        if i in live and length and what != "commit":
            a = ref.bounds(want[i, :length], want_mass[i, :length], xt, xt, dk, T)
            worst[0] = max(worst[0], ref.check(mine, want[i, :length].cpu(), a.cpu(), f"out of row {i}"))
            (view[at:at + length] if packed else view[i]).fill_(POISON)
        at += length
    assert (untouched == POISON).all(), "out written where it must not be"
    for i in live:
        slot = int(slots[i])
        if what != "verify":
            a = ref.bounds(last[i], last_mass[i], st, xt, dk, T)
            worst[1] = max(worst[1], ref.check(pool[slot], last[i].cpu(), a.cpu(), f"state of row {i}"))
            pool[slot] = before[slot, :hv * dk * dv].unflatten(0, (hv, dk, dv))
    assert torch.equal(pool_full, before), "pool written where it must not be"
    return what, pair, (n, T, hq, hv, dk, dv), worst


@pytest.mark.parametrize("seed", range(60))
def test_prompts(seed):
    _say("sweep, prompts", seed)
    rng, gen = random.Random(seed), torch.Generator().manual_seed(seed)
    _say(*_run(rng, gen, True))


@pytest.mark.parametrize("seed", range(100))
def test_few_tokens(seed):
    _say("sweep, few tokens", seed)
    rng, gen = random.Random(1000 + seed), torch.Generator().manual_seed(1000 + seed)
    _say(*_run(rng, gen, False))
