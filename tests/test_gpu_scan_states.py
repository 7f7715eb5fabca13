"""GPU tests of the selective scan for every number of states, with NaN wherever a row of B or C does not
reach: beside the rows, behind the last one (in the same allocation), and in the tokens that follow.  A
kernel that loads rows rounded up to sixteens, or to the lanes' runs, must not let any of it into an output."""

import pytest
import torch

import test_gpu_selective_scan as scan

pytestmark = pytest.mark.gpu

NAN = float("nan")
STATES = [8, 16, 24, 32, 40, 48, 56, 64]
# what is called, tokens of each row, and whether the prompts' rows are cut
CALLS = {"prompts": ("prefill", [1, 18, 0, 33, 4]), "cut": ("prefill", [700, 3]), "update3": ("update", [3] * 3),
         "verify4": ("verify", [4] * 3), "verify9": ("verify", [9] * 3), "update32": ("update", [32] * 2)}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from causal_conv1d_verify_amd import _seqops

    _seqops.load()


def _problem(call, n, pair, seed=1):
    kind, lengths = CALLS[call]
    packed = kind == "prefill"
    p = scan.Problem(lengths, 40, n, pair, packed=packed, T=None if packed else lengths[0], seed=seed)
    return kind, p


def _call(kind, p):
    import causal_conv1d_verify_amd as cv

    if kind == "prefill":
        if max(p.lengths) > 600:
            info = cv.selective_scan_describe("prefill", p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, p.cu, max_len=p.T, **p.kw())
            assert info.segment_tokens > 0
        scan.prefill(p)
    else:
        getattr(cv, "selective_scan_" + kind)(p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, **p.kw())


def _place(p, gap):
    """B and C as rows of one buffer of NaN, `gap` NaNs behind each, and two more rows of NaN behind the last;
    gap None: each a contiguous tensor of its own in such a buffer."""
    tokens, n = p.tokens, p.n
    lead = p.x.shape[:-1]

    def of(name, view):
        view.copy_(getattr(p, name).reshape(tokens, n))
        setattr(p, name, view.unflatten(0, lead) if len(lead) > 1 else view)

    if gap is None:
        for name in ("B", "C"):
            of(name, torch.full(((tokens + 2) * n + 64,), NAN, dtype=p.xt, device="cuda")[:tokens * n].view(tokens, n))
    else:
        wide = torch.full((tokens + 2, 2 * (n + gap)), NAN, dtype=p.xt, device="cuda")
        of("B", wide[:tokens, :n])
        of("C", wide[:tokens, n + gap:2 * n + gap])


@pytest.mark.parametrize("pair", scan.PAIRS)
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", STATES)
@pytest.mark.parametrize("gap", [None, 1, 24])
def test_nothing_beside_the_rows_is_used(pair, call, n, gap):
    print("[case]", pair, call, n, gap, flush=True)
    kind, p = _problem(call, n, pair)
    want = p.expect(writes=kind != "verify")
    _place(p, gap)
    _call(kind, p)
    p.check(want)


@pytest.mark.parametrize("where", ["B", "C"])
@pytest.mark.parametrize("value", [NAN, float("inf")])
@pytest.mark.parametrize("call", ["prompts", "cut", "verify9", "update3"])
@pytest.mark.parametrize("n", STATES)
def test_a_later_token_stays_out_of_earlier_ones(where, value, call, n):
    """B and C without gaps, all of one token's not finite: earlier tokens and other rows keep their bits, the
    row before it in memory among them."""
    print("[case]", where, value, call, n, flush=True)
    token = {"prompts": 19, "cut": 700, "verify9": 9, "update3": 4}[call]   # a later row's first, or second
    first, end = {"prompts": (19, 52), "cut": (700, 703), "verify9": (9, 18), "update3": (4, 6)}[call]
    outs = []
    for bad in (False, True):
        kind, p = _problem(call, n, "bf16_f32")
        _place(p, None)
        if bad:
            getattr(p, where).view(p.tokens, n)[token] = value
        _call(kind, p)
        torch.cuda.synchronize()
        outs.append(p.out.reshape(p.tokens, p.d))
    same = torch.ones(p.tokens, dtype=torch.bool)
    same[first:end if where == "B" else token + 1] = False
    assert torch.equal(outs[0][same], outs[1][same])
    assert not torch.isfinite(outs[1][token].float()).any()


@pytest.mark.parametrize("where", ["x", "dt", "z"])
@pytest.mark.parametrize("value", [NAN, float("inf")])
@pytest.mark.parametrize("call", ["prompts", "cut", "verify9", "update3"])
@pytest.mark.parametrize("n", STATES)
def test_a_channel_stays_out_of_the_others(where, value, call, n):
    """x, dt or z of one channel of a later token: its own channel from there on (z: there) alone."""
    print("[case]", where, value, call, n, flush=True)
    token = {"prompts": 30, "cut": 350, "verify9": 13, "update3": 4}[call]
    end = {"prompts": 52, "cut": 700, "verify9": 18, "update3": 6}[call]
    outs = []
    for bad in (False, True):
        kind, p = _problem(call, n, "bf16_f32")
        _place(p, None)
        if bad:
            t = getattr(p, where)
            t[(token,) if t.dim() == 2 else (token // p.T, token % p.T)][21] = value
        _call(kind, p)
        torch.cuda.synchronize()
        outs.append(p.out.reshape(p.tokens, p.d))
    same = torch.ones(p.tokens, p.d, dtype=torch.bool)
    same[token:token + 1 if where == "z" else end, 21] = False
    assert torch.equal(outs[0][same], outs[1][same])
    assert not torch.isfinite(outs[1][token, 21].float())
