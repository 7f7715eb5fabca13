"""When prompts are cut into segments, seen from the host: a call without a workspace is not cut."""

import os

import pytest

from causal_conv1d_verify_amd import _lib as base
from causal_conv1d_verify_amd import _linattn as la


def _workspace(n_seq, tokens, T, heads=4, dk=64, dv=64, x=base.CV_BF16, state=base.CV_F32, n_slots=None):
    if not os.path.exists(la.LIB_PATH):
        pytest.skip("liblinattn.so not built (run __graft_entry__.build())")
    lib = la.load()
    s = la.LaShape(n_seq, T, heads, heads, dk, dv, 0.1, x, state, n_seq if n_slots is None else n_slots,
                   0, dk * heads, dk, 0, dk * heads, dk, 0, dv * heads, dv, 0, dv * heads, dv, 0, heads,
                   heads * dk * dv, tokens)
    need = lib.linattn_prefill_workspace(s)
    assert need >= 0, lib.linattn_last_error()
    return need


@pytest.mark.parametrize("x", [base.CV_BF16, base.CV_F32])
@pytest.mark.parametrize("T", [100, 512, 8192, 2 ** 31 - 1])
def test_a_loose_bound_cuts_nothing(T, x):
    """No row is longer than all tokens together, whatever max_len says."""
    assert _workspace(1, 100, T, x=x) == 0
    assert _workspace(8, 200, T, x=x) == 0


@pytest.mark.parametrize("x", [base.CV_BF16, base.CV_F32])
@pytest.mark.parametrize("T", [4000, 8192, 2 ** 31 - 1])
def test_a_long_row_is_cut_under_any_bound(T, x):
    tight = _workspace(2, 4000, 4000, x=x)
    assert tight > 0 and _workspace(2, 4000, T, x=x) == tight


def test_cuts_keep_every_launch_within_a_grid():
    """Rows times heads within a launch, times the pieces of a state not: the second of three
    launches would be refused with the first one under way."""
    big = dict(heads=64, dk=256, dv=256, n_slots=1)
    assert _workspace(1 << 18, 1 << 20, 1 << 20, **big) > 0
    assert _workspace(1 << 20, 1 << 21, 1 << 20, **big) == 0


@pytest.mark.parametrize("x", [base.CV_BF16, base.CV_F32])
def test_rows_that_are_not_cut_take_no_workspace(x):
    """A long prompt among short ones: all tokens together make at most 512 segments of a head's tile,
    and cut rows' last ones as many again, however many rows there are."""
    heads, dk, dv = 48, 128, 128
    most = 2 * 512 * dk * dv * 4                 # tiles of 128 columns at most

    def need(n_seq, tokens):
        return _workspace(n_seq, tokens, 16384, heads=heads, dk=dk, dv=dv, x=x)

    assert 0 < need(1, 16384) <= need(256, 16384 + 255 * 160) <= most + 8192
    assert need(20000, 16384 + 19999) <= most + 8192
