"""GPU tests of the selective scan at the ends of its rates of decay: A up to fp32's lowest value, whose state
keeps nothing of the tokens before and everything where a step is nothing at all, and A of 0, whose state
keeps everything whatever the steps."""

import pytest
import torch

import test_gpu_selective_scan as scan

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min
CALLS = {"prompts": ("prefill", [5, 18, 0, 33, 1]), "cut": ("prefill", [700, 3]), "update1": ("update", [1] * 3),
         "update3": ("update", [3] * 3), "verify9": ("verify", [9] * 3), "commit": ("commit", [6] * 3)}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from causal_conv1d_verify_amd import _seqops

    _seqops.load()


def _run(call, n, pair, change, softplus):
    import causal_conv1d_verify_amd as cv

    kind, lengths = CALLS[call]
    packed = kind == "prefill"
    p = scan.Problem(lengths, 40, n, pair, packed=packed, T=None if packed else lengths[0], bias=False, softplus=softplus, seed=n)
    change(p)
    if kind == "commit":
        num = torch.tensor([6, 0, 4], dtype=torch.int32)
        want = p.expect(taken=num, outputs=False)
        cv.selective_scan_commit(p.x, p.dt, p.A, p.B, p.pool, num.cuda(), **p.kw(out=False))
    else:
        want = p.expect(writes=kind != "verify")
        if packed:
            scan.prefill(p)
        else:
            getattr(cv, "selective_scan_" + kind)(p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, **p.kw())
    p.check(want)
    torch.cuda.synchronize()
    assert torch.isfinite(p.pool_full.float()).all() and torch.isfinite(p.out_full.float()).all()


@pytest.mark.parametrize("pair", scan.PAIRS)
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", [8, 16, 24, 64])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lowest", [LOWEST, -2.4e38])
def test_rates_of_the_lowest_value(pair, call, n, softplus, lowest):
    """Some channels' steps are nothing (softplus of -200 is 0 in fp32), and some tokens' of all."""
    print("[case]", pair, call, n, softplus, lowest, flush=True)

    def change(p):
        p.A[:, ::3] = lowest
        p.A[::5] = lowest
        nothing = -200.0 if softplus else 0.0
        p.dt[..., ::4] = nothing
        p.dt.view(-1, p.d)[::2] = nothing

    _run(call, n, pair, change, softplus)


@pytest.mark.parametrize("pair", ["f32", "bf16_f32"])
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", [8, 16, 24, 64])
@pytest.mark.parametrize("softplus", [True, False])
def test_rates_of_zero(pair, call, n, softplus):
    """Steps whose sum passes fp32's range over tokens that add nothing, then ordinary ones."""
    print("[case]", pair, call, n, softplus, flush=True)

    def change(p):
        p.A[:, 1::3] = 0.0
        p.A[7] = 0.0
        far = torch.arange(p.tokens, device="cuda") % 100 < 60
        dt, x = p.dt.view(-1, p.d), p.x.view(-1, p.d)
        dt[far] = 1e38
        x[far] = 0.0

    _run(call, n, pair, change, softplus)
