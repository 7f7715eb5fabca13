"""The token that accept_drafts draws has a weight, also where rounding decides which it is: sums of weights in
two orders that differ by their last bit, with nothing behind the place where they do."""

import pytest
import torch

pytestmark = pytest.mark.gpu

PART = 1024      # weights that the kernel sums first


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from causal_conv1d_verify_amd import _seqops

    _seqops.load()


def _lane_sums(v):
    """The running sums over 16 lanes, each adding the lane 1, 2, 4 and 8 before it."""
    s = list(v)
    for step in (1, 2, 4, 8):
        s = [x + (s[i - step] if i >= step else 0.0) for i, x in enumerate(s)]
    return s


def _weights(lanes):
    """1/2 and two of 2^-54, in lanes 0 to 2; nothing in lanes 3 and 4; 1/2 in lane 5.  In order the first three
    make 1/2 (each tie rounds to even); the lanes' sum of the second and third is added to 1/2 as a whole."""
    v = [0.5, 2.0 ** -54, 2.0 ** -54, 0.0, 0.0, 0.5] + [0.0] * 10
    s = _lane_sums(v)
    assert (s[1] + v[2], s[2], s[15]) == (0.5, 0.5 + 2.0 ** -53, 1.0)
    target = torch.zeros(lanes * PART)
    return v, target


@pytest.mark.parametrize("parts", [1, 2, 16], ids=lambda p: f"{p}-parts-a-lane")
@pytest.mark.parametrize("place", [0, 511, 1023])
def test_a_part_without_weights_is_passed_over(parts, place):
    """The given number's share is exactly 1/2, which lies between the two."""
    print("[case]", parts, place, flush=True)
    import causal_conv1d_verify_amd as cv

    v, target = _weights(256 * parts if parts > 1 else 16)
    for lane, w in enumerate(v):
        target[lane * parts * PART + place] = w
    tokens = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    num, nxt = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    cv.accept_drafts(tokens, target.view(1, 1, -1).cuda(), torch.tensor([[0.5]], device="cuda"), num, nxt)
    assert int(num) == 1
    # the third token exactly, the last by sums in order; both have a weight
    assert int(nxt) in [lane * parts * PART + place for lane in (2, 5)]
    assert target[int(nxt)] > 0


@pytest.mark.parametrize("seed", range(20))
def test_truncated_probabilities(seed):
    """Of most rows a few tokens are left, of very different weights, in parts with others that are empty."""
    print("[case]", seed, flush=True)
    import causal_conv1d_verify_amd as cv

    gen = torch.Generator().manual_seed(seed)
    n, V = 64, 40 * PART + 17
    target = torch.zeros(n, 1, V)
    at = torch.randint(0, V, (n, 1, 24), generator=gen)
    target.scatter_(2, at, 2.0 ** (-60 * torch.rand(n, 1, 24, generator=gen)))
    num, nxt = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    cv.accept_drafts(torch.zeros(n, 1, dtype=torch.int32, device="cuda"), target.cuda(), torch.rand(n, 1, generator=gen).cuda(), num, nxt)
    nxt = nxt.cpu().long()
    assert bool((nxt >= 0).all()) and bool((target[torch.arange(n), 0, nxt] > 0).all())
