"""The commit of a tree's accepted tokens: accept_drafts' path gathers them to the front of their rows, from
where the commits of the scan and of linear attention fold them.  Against the 64-bit recurrences over the path
that the 64-bit verdict names."""

import pytest
import torch

import linear_reference
import sequence_reference as ref
import test_gpu_accept as accept

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from causal_conv1d_verify_amd import _seqops

    _seqops.load()


def _along(t, path):
    """[n, T, ...] rows in the order of path; places behind its end are the first, which no commit folds."""
    at = path.long().clamp(min=0).view(*path.shape, *[1] * (t.dim() - 2))
    return t.gather(1, at.expand_as(t)).contiguous()


@pytest.mark.parametrize("n,T,pads", [(1, 2, ()), (12, 7, (3,)), (40, 17, (0, 39)), (6, 32, ())])
def test_states_behind_an_accepted_path(n, T, pads):
    print("[case] tree commit", n, T, flush=True)
    import causal_conv1d_verify_amd as cv

    tree = accept.Problem(n, T, 60, "tree", seed=T, sharp=5.0, pads=pads)
    num, _, _, path = tree.expect()
    tree.gpu()
    tree.out[0].fill_(0)                           # (rows that are skipped commit nothing)
    tree.call()
    assert any(int(num[i]) > 1 and not torch.equal(path[i, :num[i]], torch.arange(int(num[i]), dtype=torch.int32))
               for i in range(n) if tree.slots[i] >= 0) or n == 1
    gen = torch.Generator().manual_seed(n)
    slots = tree.slots.cuda()
    along = tree.path[:, :T].contiguous()

    # ---- the scan
    d, N = 72, 16
    x, dt, B = (torch.randn(n, T, w, generator=gen).to(BF16) for w in (d, d, N))
    A, first = -torch.rand(d, N, generator=gen) * 4, torch.randn(n, d, N, generator=gen)
    state = first.cuda()
    cv.selective_scan_commit(*(_along(t.cuda(), along) for t in (x, dt)), A.cuda(), _along(B.cuda(), along), state, tree.out[0],
                             slot_idx=slots)
    # ---- linear attention
    H, dk = 3, 64
    k, v = (torch.randn(n, T, H, dk, generator=gen).to(BF16) for _ in range(2))
    g, S0 = -torch.rand(n, T, H, generator=gen), torch.randn(n, H, dk, dk, generator=gen)
    S = S0.cuda()
    cv.linear_attn_commit(*(_along(t.cuda(), along) for t in (k, v)), _along(g.cuda(), along), S, tree.out[0], slot_idx=slots)
    torch.cuda.synchronize()

    got, got_S = state.cpu(), S.cpu()
    for i in range(n):
        if tree.slots[i] < 0:
            assert torch.equal(got[i], first[i]) and torch.equal(got_S[i], S0[i])
            continue
        way = path[i, :num[i]].long()
        row = ref.Scan(first[i], A)
        for t in way:
            row.token(x[i, t], dt[i, t], B[i, t])
        h, tol = row.state()
        assert bool(((got[i].double() - h).abs() <= ref.rounded(h, tol, torch.float32)).all())
        one = slice(i, i + 1)
        _, last, _, mass = linear_reference.recurrence(*(t[one][:, way] for t in (k, k, v, g)), S0[one], 1.0)
        linear_reference.check(got_S[one], last, linear_reference.bounds(last, mass, torch.float32, BF16, dk, T), "linear attention")
