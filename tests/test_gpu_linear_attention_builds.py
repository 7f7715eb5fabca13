"""GPU tests of the kernels of few tokens in every build that a call can get, each asking first which
one it is: blocks of rows and of tokens of the matrix form, row groups and tile widths of the
recurrence.  Bounds and problems are those of test_gpu_linear_attention.py.
"""

import pytest
import torch

import linear_reference as ref
from test_gpu_linear_attention import BF16, F32, PAIRS, Problem, _need_gpu, _say  # noqa: F401

pytestmark = pytest.mark.gpu


def _info(p, name):
    import causal_conv1d_verify_amd as cv

    args = (p.k, p.v, p.g, p.pool) if name == "commit" else (p.q, p.k, p.v, p.g, p.pool, p.out)
    return cv.linear_attn_describe(name, *args, slot_idx=p.slot_idx)


def _run(p):
    """Update, then verify and commit of some, of one problem against the recurrence."""
    import causal_conv1d_verify_amd as cv

    want = p.expected()
    cv.linear_attn_update(p.q, p.k, p.v, p.g, p.pool, p.out, slot_idx=p.slot_idx)
    torch.cuda.synchronize()
    p.check(want)
    p.pool_full.copy_(p.before)
    p.out_full.fill_(7.25)
    cv.linear_attn_verify(p.q, p.k, p.v, p.g, p.pool, p.out, slot_idx=p.slot_idx)
    torch.cuda.synchronize()
    p.check(want, state=False)
    counts = [(3 * i + 1) % (p.T + 1) for i in range(p.n)]
    some = p.expected(counts=counts)
    cv.linear_attn_commit(p.k, p.v, p.g, p.pool, torch.tensor(counts, dtype=torch.int32, device="cuda"),
                          slot_idx=p.slot_idx)
    torch.cuda.synchronize()
    p.check((want[0], some[1], want[2], some[3]))


@pytest.mark.parametrize("pair", ["bf16", "bf16_f32"])
@pytest.mark.parametrize("T", [2, 16, 17, 32])
@pytest.mark.parametrize("heads", [(64, 128), (128, 128), (96, 200), (72, 64), (136, 256), (256, 72)], ids=str)
def test_matrix_form(heads, T, pair):
    from causal_conv1d_verify_amd import _linattn as la

    _say("matrix form", heads, T, pair)
    p = Problem([T] * 3, 2, 4, *heads, pair, packed=False, T=T, pads=(1,))
    for name in ("update", "verify", "commit"):
        assert _info(p, name).kernel == la.LA_KERNEL_FEW
    _run(p)


@pytest.mark.parametrize("T", [1, 7])
@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("wide", [False, True])
def test_recurrence_of_fp32(wide, dk, T):
    """Tiles of 32 columns below 512 workgroups, of 64 from there on."""
    from causal_conv1d_verify_amd import _linattn as la

    _say("recurrence", wide, dk, T)
    n = 65 if wide else 5
    p = Problem([T] * n, 2, 4, dk, 72, "f32", packed=False, T=T, pads=(1,))
    for name in ("update", "verify", "commit"):
        info = _info(p, name)
        assert info.kernel == la.LA_KERNEL_TOKENS and info.state_cols == (64 if wide else 32)
    _run(p)


@pytest.mark.parametrize("dk", [40, 128, 200])
@pytest.mark.parametrize("pair", ["bf16", "bf16_f32"])
def test_recurrence_of_single_bf16_tokens(pair, dk):
    from causal_conv1d_verify_amd import _linattn as la

    _say("single tokens", pair, dk)
    p = Problem([1] * 6, 3, 6, dk, 136, pair, packed=False, T=1, pads=(4,))
    info = _info(p, "update")
    assert info.kernel == la.LA_KERNEL_TOKENS and info.state_cols == (64 if pair == "bf16" else 32)
    _run(p)


@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("pair", PAIRS)
def test_recurrence_of_prompts_far_apart_on_a_full_card(pair, dk):
    """Tokens 2^24 elements apart in 512 heads: the wide tiles of every type."""
    import causal_conv1d_verify_amd as cv
    from causal_conv1d_verify_amd import _linattn as la

    _say("far apart, many heads", pair, dk)
    xt, st = PAIRS[pair]
    gen = ref.spread(dk, 12)
    T, hq, hv, dv, far = 3, 2, 512, 24, 1 << 24
    host = torch.randn(T, 2 * hq * dk + hv * dv, generator=gen).to(xt)
    rows = torch.zeros(T * far, dtype=xt, device="cuda").as_strided((T, host.shape[1]), (far, 1))
    rows.copy_(host)

    def heads(t):
        return (t[:, :hq * dk].unflatten(1, (hq, dk)), t[:, hq * dk:2 * hq * dk].unflatten(1, (hq, dk)),
                t[:, 2 * hq * dk:].unflatten(1, (hv, dv)))

    pool, g = torch.randn(1, hv, dk, dv, generator=gen).to(st), ref.log_decays((T, hv), gen)
    want = ref.recurrence(*(t[None] for t in heads(host)), g[None], pool, ref.scale_of(dk))
    S, out = pool.cuda(), torch.zeros(T, hv, dv, dtype=xt, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    args = (*heads(rows), g.cuda(), S, out, cu)
    info = cv.linear_attn_describe("prefill", *args, max_len=T)
    assert info.kernel == la.LA_KERNEL_TOKENS and info.state_cols == (128 if st == BF16 else 64)
    cv.linear_attn_prefill(*args, max_len=T)
    torch.cuda.synchronize()
    ref.check(out[None], want[0], ref.bounds(want[0], want[2], xt, xt, dk, T), "out")
    ref.check(S, want[1], ref.bounds(want[1], want[3], st, xt, dk, T), "state")


@pytest.mark.parametrize("heads", [(64, 72), (96, 64), (128, 136), (192, 40), (256, 128)], ids=str)
@pytest.mark.parametrize("T", [12, 16, 32])
def test_chunks_of_fp32(T, heads):
    from causal_conv1d_verify_amd import _linattn as la

    _say("one chunk", T, heads)
    p = Problem([T] * 3, 1, 2, *heads, "f32", packed=False, T=T, pads=(1,))
    assert _info(p, "verify").kernel == la.LA_KERNEL_CHUNKED_F32
    assert _info(p, "commit").kernel == (la.LA_KERNEL_CHUNKED_F32 if T >= 16 else la.LA_KERNEL_TOKENS)
    _run(p)
