"""GPU tests of rows that are cut into segments, which are workgroups in no order: every segment
starts from the state that the call found, whenever the row's last one writes the pool.  Bounds and
problems are those of test_gpu_linear_attention.py, the recurrence in 64 bits runs on the GPU.
"""

import pytest
import torch

import linear_reference as ref
from test_gpu_linear_attention import BF16, F32, Problem, _need_gpu, _say  # noqa: F401

pytestmark = pytest.mark.gpu


def _expected(p):
    g = p.g
    if g is not None and g.dim() == 1:           # a decay for each token, which moves with its rows
        p.g = g.expand(p.starts[-1], p.hv)
    with torch.device("cuda"):
        want = p.expected()
    p.g = g
    return [t.cpu() for t in want]


def _segment(p, chunk, tiles):
    """Tokens of a segment, by the rule of la_api.cpp: a 512th of all chunks, 4 at least."""
    return chunk * max(4, (sum(p.lengths) // chunk + 1) * p.hv * tiles // 512)


def _bytes(p):
    """The workspace that the call asks for: none where no row is cut."""
    from causal_conv1d_verify_amd import linear_attention as m

    lib, _, _, args, _ = m._attn_args("prefill", p.q, p.k, p.v, p.g, p.pool, p.out, cu_seqlens=p.cu,
                                      max_len=p.T, slot_idx=p.slot_idx)
    return lib.linattn_prefill_workspace(args[0])


# pair, rows, tokens, q heads, v heads, dk, dv, chunk, tiles of a head: 768 workgroups, of which the
# card holds 512; the last segment of each row is a single token and done long before the others
CASES = [("bf16_f32", 4, 1025, 4, 64, 128, 128, 64, 1),
         ("bf16", 4, 1025, 4, 64, 128, 128, 64, 1),
         ("f32", 4, 1025, 4, 32, 256, 128, 32, 2)]


@pytest.mark.parametrize("decay", ["none", "head"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: c[0])
def test_segments_start_from_the_state_that_the_call_found(case, decay):
    pair, n, T, hq, hv, dk, dv, chunk, tiles = case
    _say("segments, one token last", case, decay)
    p = Problem([T] * n, hq, hv, dk, dv, pair, packed=True, decay=decay, started=[1, 1, 0, 1])
    length = _segment(p, chunk, tiles)
    assert T % length == 1 and T > 2 * length and _bytes(p) > 0
    want = _expected(p)
    p.prefill()
    p.check(want)
    first = p.out_full.clone(), p.pool_full.clone()
    for _ in range(4):
        p.pool_full.copy_(p.before)
        p.prefill()
        assert torch.equal(first[0], p.out_full) and torch.equal(first[1], p.pool_full)


@pytest.mark.parametrize("pair", ["bf16_f32", "bf16", "f32"])
def test_segments_beside_other_work(pair):
    """Another stream holds compute units while the segments run."""
    _say("segments beside other work", pair)
    p = Problem([3000, 1, 1537, 0, 700], 1, 8, 64, 64, pair, packed=True, started=[1, 1, 1, 1, 0])
    assert _bytes(p) > 0
    want = _expected(p)
    p.prefill()
    p.check(want)
    first = p.out_full.clone(), p.pool_full.clone()
    other, a = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        p.pool_full.copy_(p.before)
        with torch.cuda.stream(other):
            b = a @ a
        p.prefill()
        other.synchronize()
        assert torch.equal(first[0], p.out_full) and torch.equal(first[1], p.pool_full)
    assert b.shape == a.shape


@pytest.mark.parametrize("pair", ["bf16_f32", "f32"])
def test_first_states_of_cut_rows_that_are_not_finite(pair):
    """A first state of inf reaches its own row's outputs and state, from its column on; behind a
    decay of exp(-inf) = 0 it is NaN, as 0 * inf is."""
    _say("first state not finite", pair)
    p = Problem([2100, 1500], 1, 2, 64, 64, pair, packed=True, decay="head")
    assert _bytes(p) > 0
    want = _expected(p)
    slot = int(p.slots[0])
    p.pool[slot, 1, :, 5] = float("inf")
    p.prefill()
    got, pool = p.out.cpu(), p.pool.cpu()
    assert not torch.isfinite(got[:p.lengths[0], 1, 5]).any()
    assert not torch.isfinite(pool[slot, 1, :, 5]).any()
    keep = [c for c in range(64) if c != 5]
    for i in (0, 1):
        at = slice(p.starts[i], p.starts[i] + p.lengths[i])
        a = ref.bounds(want[0][i, :p.lengths[i]], want[2][i, :p.lengths[i]], p.xt, p.xt, p.dk, p.T)
        ref.check(got[at][..., keep], want[0][i, :p.lengths[i]][..., keep], a[..., keep], f"row {i}")
        a = ref.bounds(want[1][i], want[3][i], p.st, p.xt, p.dk, p.T)
        ref.check(pool[int(p.slots[i])][..., keep], want[1][i][..., keep], a[..., keep], f"state {i}")
