"""Seeded random problems over the argument space of the selective scan, the rotation and the verdict,
against the 64-bit forms; each names itself before it runs."""

import random

import pytest
import torch

import test_gpu_accept as accept
import test_gpu_rotary as rotary
import test_gpu_selective_scan as scan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(60))
def test_scans(seed):
    import causal_conv1d_verify_amd as cv

    rng = random.Random(seed)
    kind = rng.choice(["prefill", "prefill", "update", "verify", "commit"])
    n, d = 8 * rng.randint(1, 8), 8 * _log(rng, 1, 40)
    rows = _log(rng, 1, 12)
    common = dict(gate=rng.random() < 0.7, skip=rng.random() < 0.7, bias=rng.random() < 0.7, softplus=rng.random() < 0.8,
                  pads=tuple(i for i in range(rows) if rng.random() < 0.15), seed=seed, off=rng.randint(0, 9))
    if not common["softplus"]:
        common["bias"] = False                     # (its rates would grow)
    pair = rng.choice(sorted(scan.PAIRS))
    if kind == "prefill":
        top = _log(rng, 1, 900)
        lengths = [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(rows)]
        print("[case]", seed, kind, lengths, d, n, pair, common, flush=True)
        p = scan.Problem(lengths, d, n, pair, packed=True, started=rng.choice([None, [rng.randint(0, 1) for _ in lengths]]), **common)
        want = p.expect()
        scan.prefill(p)
    else:
        T = rng.randint(1, 32)
        print("[case]", seed, kind, T, rows, d, n, pair, common, flush=True)
        p = scan.Problem([T] * rows, d, n, pair, packed=False, T=T, **common)
        if kind == "commit":
            num = torch.tensor([rng.randint(0, T) for _ in range(rows)], dtype=torch.int32)
            want = p.expect(taken=num, outputs=False)
            cv.selective_scan_commit(p.x, p.dt, p.A, p.B, p.pool, num.cuda(), **p.kw(out=False))
        else:
            want = p.expect(writes=kind == "update")
            getattr(cv, "selective_scan_" + kind)(p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, **p.kw())
    p.check(want)


@pytest.mark.parametrize("seed", range(60))
def test_heads(seed):
    rng = random.Random(1000 + seed)
    dim = 16 * rng.randint(1, 16)
    rot = rng.choice([dim, 16 * rng.randint(0, dim // 16)])
    args = (_log(rng, 1, 3000), rng.randint(1, 70), rng.randint(0, 20), dim, rot, rng.choice([torch.float32, torch.bfloat16]))
    if args[0] * (args[1] + args[2]) * dim > 4e6:
        args = (rng.randint(1, 40), *args[1:])
    kw = dict(norm=(rng.random() < 0.7, rng.random() < 0.7), first=rng.choice([0, _log(rng, 1, 2 ** 30)]), wide=rng.random() < 0.5)
    interleaved = rng.random() < 0.5
    print("[case]", seed, args, kw, interleaved, flush=True)
    p = rotary.Problem(*args, seed=seed, **kw)
    want = p.expect(interleaved)
    p.call(interleaved=interleaved)
    p.check(want)


@pytest.mark.parametrize("seed", range(80))
def test_verdicts(seed):
    rng = random.Random(2000 + seed)
    n, T, vocab = _log(rng, 1, 60), rng.randint(1, 32), _log(rng, 1, 20000)
    while n * T * vocab > 3e6:
        n, vocab = max(1, n // 2), max(1, vocab // 2)
    kind, dtype = rng.choice(["chain", "certain", "tree"]), rng.choice([torch.float32, torch.bfloat16])
    print("[case]", seed, n, T, vocab, kind, dtype, flush=True)
    p = accept.Problem(n, T, vocab, kind, dtype, seed=seed, sharp=rng.choice([0.5, 2.0, 5.0]), near=rng.choice([0.2, 1.0]),
                       pads=tuple(i for i in range(n) if rng.random() < 0.1))
    gen = torch.Generator().manual_seed(seed)
    p.tokens = torch.where(torch.rand(n, T, generator=gen) < 0.1, torch.full_like(p.tokens, -1), p.tokens)
    if kind == "tree":
        p.parent[:, 1:] = torch.where(torch.rand(n, T - 1, generator=gen) < 0.1, torch.full_like(p.parent[:, 1:], -1), p.parent[:, 1:])
    p.run()
