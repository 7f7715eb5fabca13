"""Which strides of a packed `out` are taken: its elements have to be apart for the tokens that there
are, whatever bound on a row's length the call names.  Host side only: the size of the workspace is
asked for, which validates the shape and launches nothing."""

import os

import pytest

from causal_conv1d_verify_amd import _lib as base
from causal_conv1d_verify_amd import _linattn as la

HEADS, DV = 4, 64


def _refused(tokens, T, tok, head, n_seq=2, heads=HEADS):
    if not os.path.exists(la.LIB_PATH):
        pytest.skip("liblinattn.so not built (run __graft_entry__.build())")
    lib = la.load()
    s = la.LaShape(n_seq, T, heads, heads, 64, DV, 0.1, base.CV_BF16, base.CV_F32, n_seq, 0,
                   64 * heads, 64, 0, 64 * heads, 64, 0, DV * heads, DV, 0, tok, head, 0, heads,
                   heads * 64 * DV, tokens)
    rc = lib.linattn_prefill_workspace(s)
    assert rc >= 0 or (rc == base.CV_EINVAL and b"overlap" in lib.linattn_last_error())
    return rc < 0


@pytest.mark.parametrize("T", [1, 2, 16, 100, 299, 300, 512, 1 << 20])
def test_what_is_apart_is_taken(T):
    assert not _refused(300, T, HEADS * DV, DV)             # [total, heads, dv]
    assert not _refused(300, T, HEADS * DV + 8, DV)
    assert not _refused(300, T, DV, 300 * DV)               # [heads, total, dv]
    assert not _refused(300, T, DV, 304 * DV)
    assert not _refused(1, T, 0, DV)                        # one token: its stride is of no account
    assert not _refused(300, T, DV, 0, heads=1)
    assert not _refused(0, T, HEADS * DV, DV)               # a number that is not known
    assert not _refused(0, T, DV, 300 * DV)


@pytest.mark.parametrize("T", [1, 2, 16, 100, 299, 300, 512, 1 << 20])
def test_what_overlaps_is_refused(T):
    assert _refused(300, T, 0, DV)
    assert _refused(300, T, DV, 100 * DV)
    assert _refused(300, T, DV, 299 * DV)
    assert _refused(300, T, HEADS * DV - 8, DV)
    assert _refused(2, T, HEADS * DV - 8, DV)
    assert _refused(300, T, HEADS * DV, 0)
    assert _refused(1, T, HEADS * DV, DV - 8)
    assert _refused(0, T, 0, DV)
    assert _refused(0, T, HEADS * DV - 8, DV)
    assert _refused(0, T, DV, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("max_len", [64, 2048])
def test_one_token_and_heads_before_tokens(max_len):
    """Through the binding: a prompt of a single token, and out as [heads, total, dv], under a bound
    that is longer than they are."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import causal_conv1d_verify_amd as cv
    import linear_reference as ref

    print("[case] out strides", max_len, flush=True)
    gen = ref.spread(max_len, 11)
    for T in (1, 50):
        q, k = (torch.randn(T, 2, 64, generator=gen).to(torch.bfloat16) for _ in range(2))
        v = torch.randn(T, HEADS, DV, generator=gen).to(torch.bfloat16)
        state = torch.randn(1, HEADS, 64, DV, generator=gen)
        want = ref.recurrence(q[None], k[None], v[None], torch.zeros(1, T, HEADS), state, ref.scale_of(64))
        S, out = state.cuda(), torch.zeros(HEADS, T, DV, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        cv.linear_attn_prefill(q.cuda(), k.cuda(), v.cuda(), None, S, out, cu, max_len=max_len)
        torch.cuda.synchronize()
        ref.check(out[None], want[0], ref.bounds(want[0], want[2], torch.bfloat16, torch.bfloat16, 64, T), "out")
        ref.check(S, want[1], ref.bounds(want[1], want[3], torch.float32, torch.bfloat16, 64, T), "state")
