"""GPU tests of the prompts' 128-column kernel, each asking first whether it is what runs: every row
count of the state, partial tiles, segments, and values that are not finite, which have to stay in
their own column.  Bounds and problems are those of test_gpu_linear_attention.py.
"""

import math

import pytest
import torch

import linear_reference as ref
from test_gpu_linear_attention import BF16, Problem, _need_gpu, _say  # noqa: F401
from test_gpu_linear_attention_segments import _expected

pytestmark = pytest.mark.gpu

SHAPES = [(64, 128), (40, 72), (128, 128), (128, 72), (72, 136), (192, 128), (136, 200), (256, 256), (200, 248),
          (256, 72)]
MANY = [65, 130, 3, 64, 0, 129, 1, 200]          # cycled over rows


def _wide(p, cut):
    """The call's kernel has 128 columns, and cuts rows or not."""
    import causal_conv1d_verify_amd as cv
    from causal_conv1d_verify_amd import _linattn as la

    info = cv.linear_attn_describe("prefill", p.q, p.k, p.v, p.g, p.pool, p.out, p.cu, max_len=p.T,
                                   slot_idx=p.slot_idx)
    assert info.kernel == la.LA_KERNEL_CHUNKED and info.state_cols == 128
    assert info.launches == (3 if cut else 1)
    return info


def _many(dk, dv, pair="bf16_f32", n=66, hq=4, hv=8, **kw):
    return Problem([MANY[i % len(MANY)] for i in range(n)], hq, hv, dk, dv, pair, packed=True, **kw)


@pytest.mark.parametrize("pair", ["bf16", "bf16_f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_many_rows(shape, pair):
    _say("wide, many rows", shape, pair)
    p = _many(*shape, pair, pads=(7, 40), started=[i % 3 for i in range(66)])
    _wide(p, cut=False)
    g = p.g.cpu()
    g[5::37] = -math.inf
    g[11::41] = -1000.0
    g[20::5] = 0.0
    p.g = g.cuda()
    want = _expected(p)
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("decay", ["token", "head", "none"])
@pytest.mark.parametrize("pair", ["bf16", "bf16_f32"])
@pytest.mark.parametrize("shape", [(64, 128), (128, 136), (128, 128), (192, 128), (256, 256)], ids=str)
def test_segments(shape, pair, decay):
    _say("wide, segments", shape, pair, decay)
    p = Problem([2100, 5, 0, 1537, 700], 2, 8, *shape, pair, packed=True, decay=decay, started=[1, 1, 0, 0, 1])
    info = _wide(p, cut=True)
    assert 2100 > 2 * info.segment_tokens
    want = _expected(p)
    p.prefill()
    p.check(want)


def _check_row(p, want, i, upto=None, skip=None):
    """Row i's outputs before token `upto` (all), but for head and column `skip`."""
    n = p.lengths[i] if upto is None else upto
    got, value = p.out.cpu()[p.starts[i]:p.starts[i] + n].double(), want[0][i, :n].clone()
    a = ref.bounds(value, want[2][i, :n], p.xt, p.xt, p.dk, p.T)
    if skip is not None:
        got[:, skip[0], skip[1]] = value[:, skip[0], skip[1]]
    ref.check(got, value, a, f"row {i}")


def _check_state(p, want, i, skip=None):
    got, value = p.pool[int(p.slots[i])].cpu().double(), want[1][i].clone()
    if skip is not None:
        got[skip[0], :, skip[1]] = value[skip[0], :, skip[1]]
    ref.check(got, value, ref.bounds(value, want[3][i], p.st, p.xt, p.dk, p.T), f"state {i}")


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("pair", ["bf16", "bf16_f32"])
@pytest.mark.parametrize("shape", [(64, 128), (128, 72), (192, 136), (256, 128)], ids=str)
def test_one_value_that_is_not_finite(shape, pair, bad):
    """In another column, head and token of each row: it reaches that column's outputs from its token
    on, and nothing else."""
    _say("wide, one value", shape, pair, bad)
    dk, dv = shape
    p = _many(dk, dv, pair, hq=2)
    _wide(p, cut=False)
    want = _expected(p)
    at = {}
    for i, n in enumerate(p.lengths):
        if n:
            at[i] = (11 * i) % n, (3 * i) % p.hv, (7 * i + i // 8) % dv
            t, h, c = at[i]
            p.v[p.starts[i] + t, h, c] = bad
    p.prefill()
    out, pool = p.out.cpu(), p.pool.cpu()
    for i, (t, h, c) in at.items():
        _check_row(p, want, i, upto=t)
        _check_row(p, want, i, skip=(h, c))
        _check_state(p, want, i, skip=(h, c))
        assert not torch.isfinite(out[p.starts[i] + t:p.starts[i] + p.lengths[i], h, c]).any()
        assert not torch.isfinite(pool[int(p.slots[i]), h, :, c]).any()


@pytest.mark.parametrize("where", ["q", "k"])
@pytest.mark.parametrize("shape", [(64, 128), (128, 72), (256, 128)], ids=str)
def test_queries_and_keys_that_are_not_finite(shape, where):
    """A query reaches its own token of the heads that share it, a key those heads from its token on."""
    _say("wide, query or key", shape, where)
    p = _many(*shape, hq=2)
    _wide(p, cut=False)
    want = _expected(p)
    at = {i: (11 * i) % n for i, n in enumerate(p.lengths) if n}
    for i, t in at.items():
        getattr(p, where)[p.starts[i] + t, i % 2, (5 * i) % p.dk] = math.nan
    p.prefill()
    out, group = p.out.cpu(), p.hv // p.hq
    for i, t in at.items():
        _check_row(p, want, i, upto=t)
        hit = slice(i % 2 * group, (i % 2 + 1) * group)
        rest = [h for h in range(p.hv) if h not in range(hit.start, hit.stop)]
        own = out[p.starts[i]:p.starts[i] + p.lengths[i]]
        a = ref.bounds(want[0][i, :len(own)], want[2][i, :len(own)], p.xt, p.xt, p.dk, p.T)
        ref.check(own[:, rest], want[0][i, :len(own)][:, rest], a[:, rest], f"other heads of row {i}")
        assert not torch.isfinite(own[t, hit]).any()
        if where == "k":
            assert not torch.isfinite(own[t:, hit]).any()
        else:
            ref.check(own[t + 1:], want[0][i, t + 1:len(own)], a[t + 1:], f"behind, row {i}")
            _check_state(p, want, i)


@pytest.mark.parametrize("pair", ["bf16", "bf16_f32"])
def test_segments_and_one_value_that_is_not_finite(pair):
    """In the second segment of a row: its column from there on, through the workspace."""
    _say("wide, segments, one value", pair)
    p = Problem([2100, 1537, 700], 1, 8, 128, 128, pair, packed=True, decay="head", started=[1, 0, 1])
    info = _wide(p, cut=True)
    want = _expected(p)
    t, h, c = info.segment_tokens + 77, 5, 93
    p.v[p.starts[0] + t, h, c] = math.inf
    p.prefill()
    for i in range(3):
        _check_row(p, want, i, upto=t if i == 0 else None)
        _check_row(p, want, i, skip=(h, c) if i == 0 else None)
        _check_state(p, want, i, skip=(h, c) if i == 0 else None)
    assert not torch.isfinite(p.out[p.starts[0] + t:p.starts[0] + 2100, h, c]).any()


def test_the_same_every_time():
    _say("wide, repeats")
    for p, cut in ((_many(128, 128), False), (Problem([2100, 1537], 2, 16, 128, 128, "bf16_f32", packed=True), True)):
        _wide(p, cut)
        p.prefill()
        first = p.out_full.clone(), p.pool_full.clone()
        for _ in range(3):
            p.pool_full.copy_(p.before)
            p.prefill()
            assert torch.equal(first[0], p.out_full) and torch.equal(first[1], p.pool_full)


def test_replays_of_a_graph():
    """Rows of both kinds captured together, replayed with eager calls between."""
    _say("wide, graph")
    ps = [_many(128, 128), Problem([2100, 1537], 2, 16, 128, 128, "bf16", packed=True, seed=2)]
    for p, cut in zip(ps, (False, True)):
        _wide(p, cut)
        p.prefill()
    first = [(p.out_full.clone(), p.pool_full.clone()) for p in ps]
    import causal_conv1d_verify_amd as cv

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in ps:
            cv.linear_attn_prefill(p.q, p.k, p.v, p.g, p.pool, p.out, p.cu, max_len=p.T, slot_idx=p.slot_idx)
    for _ in range(3):
        for replay in (True, False):
            for p in ps:
                p.pool_full.copy_(p.before)
                p.out_full.fill_(7.25)
            if replay:
                graph.replay()
            else:
                for p in ps:
                    p.prefill()
            torch.cuda.synchronize()
            for p, (out, pool) in zip(ps, first):
                assert torch.equal(p.out_full, out) and torch.equal(p.pool_full, pool)
