"""GPU tests of how prompts are cut (segments of long rows, tiles of 64 and 128 columns, chunks at
and around their ends) and of states that are streamed past the caches.  Bounds and problems are
those of test_gpu_linear_attention.py.
"""

import math

import pytest
import torch

import linear_reference as ref
from test_gpu_linear_attention import BF16, PAIRS, Problem, _need_gpu, _say  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("length", [15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 129])
def test_ends_inside_chunks_and_tiles(length, pair):
    _say("ends", length, pair)
    p = Problem([length, 1, length], 1, 2, 72, 80, pair, packed=True, started=[1, 0, 0])
    want = p.expected()
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("dv", [8, 56, 64, 72, 120, 128, 136, 192, 256])
@pytest.mark.parametrize("dk", [8, 64, 72, 136, 200, 256])
def test_tiles_of_every_width(dk, dv, pair):
    _say("tiles", dk, dv, pair)
    p = Problem([70, 0, 33], 2, 2, dk, dv, pair, packed=True)
    want = p.expected()
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("pair", PAIRS)
def test_wide_tiles_of_many_rows(pair):
    """Enough workgroups for the 128-column tiles, with decays from none to -inf among them."""
    _say("wide", pair)
    p = Problem([65, 130, 3, 64] * 10, 1, 4, 64, 128, pair, packed=True, pads=(7,))
    g = p.g.cpu()
    g[5::37] = -math.inf
    g[11::41] = -1000.0
    g[20::5] = 0.0
    p.g = g.cuda()
    want = p.expected()
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_wide_tiles_and_values_that_are_not_finite(where, bad):
    """In each 16-token tile of a chunk: tokens before the value's own stay as they are."""
    _say("wide, not finite", where, bad)
    n = 40
    p = Problem([100] * n, 1, 4, 64, 128, "bf16_f32", packed=True)
    want = p.expected()
    at = [(7 * i) % 100 for i in range(n)]
    for i in range(n):
        getattr(p, where)[p.starts[i] + at[i]] = bad
    p.prefill()
    got = p.out.cpu()
    for i in range(n):
        a = ref.bounds(want[0][i, :at[i]], want[2][i, :at[i]], p.xt, p.xt, p.dk, p.T)
        ref.check(got[p.starts[i]:p.starts[i] + at[i]], want[0][i, :at[i]], a, f"row {i}")
        own = got[p.starts[i] + at[i]:p.starts[i] + 100]
        assert not torch.isfinite(own[:1] if where == "q" else own).any()


@pytest.mark.parametrize("pair", PAIRS)
def test_one_long_row_among_many_short_ones(pair):
    """Segments are found among 300 rows (more than a workgroup's lanes), short, empty and padded."""
    _say("long among short", pair)
    lengths = [(3 * i) % 7 for i in range(300)]
    lengths[280] = 3000
    lengths[17] = 700
    p = Problem(lengths, 1, 1, 32, 40, pair, packed=True, pads=(5, 281, 299),
                started=[i % 2 for i in range(300)])
    want = p.expected()
    p.prefill()
    p.check(want)


def test_segments_with_strong_decays_and_no_start():
    _say("segments, strong decays")
    p = Problem([2500, 1800], 1, 1, 64, 64, "bf16_f32", packed=True, started=[0, 1])
    g = p.g.cpu()
    g[700] = -math.inf
    g[1500:1600] = -300.0
    p.g = g.cuda()
    want = p.expected()
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("pair", ["f32", "bf16"])
def test_segments_and_falling_offsets(pair):
    """Offsets that fall make rows that overlap: the tokens declared are fewer than the rows hold
    together, and the rows that do not fit the workspace are left alone."""
    _say("segments, falling offsets", pair)
    p = Problem([3000, 10, 10], 1, 1, 32, 32, pair, packed=True)
    want = p.expected()
    p.cu = torch.tensor([0, 3000, 0, 3000], dtype=torch.int32, device="cuda")
    before = p.pool_full.clone()
    p.q = p.q[:3000]
    p.k, p.v, p.g, p.out = p.k[:3000], p.v[:3000], p.g[:3000], p.out[:3000]
    p.prefill()
    a = ref.bounds(want[0][0], want[2][0], p.xt, p.xt, p.dk, p.T)
    ref.check(p.out.cpu(), want[0][0], a, "out")
    slot = [int(s) for s in p.slots]
    a = ref.bounds(want[1][0], want[3][0], p.st, p.xt, p.dk, p.T)
    ref.check(p.pool[slot[0]].cpu(), want[1][0], a, "state")
    for s in slot[1:]:
        assert torch.equal(p.pool_full[s], before[s])


def test_tokens_far_apart():
    """2^24 - 8 elements from token to token: the furthest apart that go in chunks (the largest
    32-bit offsets), and 2^24, which go one by one."""
    _say("far apart")
    import causal_conv1d_verify_amd as cv

    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    gen = ref.spread(4, 9)
    T, d = 130, 32
    for far in ((1 << 24) - 8, 1 << 24):
        wide = torch.empty(T * far, dtype=BF16, device="cuda")
        qkv = wide.as_strided((T, 3, d), (far, d, 1))
        host = torch.randn(T, 3, d, generator=gen).to(BF16)
        qkv.copy_(host)
        out = wide.as_strided((T, 1, d), (far, d, 1), 4096)
        pool = torch.randn(1, 1, d, d, generator=gen)
        g = ref.log_decays((T, 1), gen)
        want = ref.recurrence(host[None, :, 0:1], host[None, :, 1:2], host[None, :, 2:3], g[None], pool,
                              ref.scale_of(d))
        pool = pool.cuda()
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        cv.linear_attn_prefill(qkv[:, 0:1], qkv[:, 1:2], qkv[:, 2:3], g.cuda(), pool, out, cu, max_len=T)
        torch.cuda.synchronize()
        ref.check(out.cpu()[None], want[0], ref.bounds(want[0], want[2], BF16, BF16, d, T), "out")
        ref.check(pool.cpu(), want[1], ref.bounds(want[1], want[3], torch.float32, BF16, d, T), "state")
        del wide, qkv, out


@pytest.mark.parametrize("name", ["linear_attn_update", "linear_attn_verify", "linear_attn_commit"])
@pytest.mark.parametrize("T", [1, 5, 20])
def test_streamed_states_are_the_same(T, name):
    """More rows than the caches keep the states of, and the same rows in two calls that they do:
    the same bits."""
    _say("streamed", T, name)
    import causal_conv1d_verify_amd as cv

    gen = torch.Generator("cuda").manual_seed(T)
    n, h, d = 36, 48, 128                        # 113 MB of fp32 states

    def randn(*shape, dtype=BF16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    q, k, v = (randn(n, T, x, d) for x in (16, 16, h))
    g = -randn(n, T, h, dtype=torch.float32).abs()
    pool = randn(n, h, d, d, dtype=torch.float32)
    slots = torch.randperm(n, device="cuda", generator=gen).to(torch.int32)
    results = []
    for pieces in (1, 2):
        S, out = pool.clone(), torch.zeros_like(v)
        for a in range(0, n, n // pieces):
            at = slice(a, a + n // pieces)
            if name == "linear_attn_commit":
                cv.linear_attn_commit(k[at], v[at], g[at], S, slot_idx=slots[at])
            else:
                getattr(cv, name)(q[at], k[at], v[at], g[at], S, out[at], slot_idx=slots[at])
        torch.cuda.synchronize()
        results.append((S, out))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert torch.equal(results[0][0], pool) == (name == "linear_attn_verify")


@pytest.mark.parametrize("shape", [(5, 1, 2, 200, 72), (3, 2, 2, 64, 256)], ids=str)
@pytest.mark.parametrize("T", [11, 12, 15, 16, 20, 32])
def test_commit_counts_and_rejected_tokens_of_a_chunk(T, shape):
    """fp32 tokens on both sides of where they go as one chunk: counts of none, some, all and out
    of range, and rejected tokens that are not finite."""
    n, hq, hv, dk, dv = shape
    _say("commit chunk", T, shape)
    import causal_conv1d_verify_amd as cv

    p = Problem([T] * n, hq, hv, dk, dv, "f32", packed=False, T=T, pads=(1,))
    counts = [T, 3, 0, T + 1, -1][:n]
    live = [i for i in range(n) if 0 <= counts[i] <= T and i != 1]
    want = p.expected(counts=[c if i in live else 0 for i, c in enumerate(counts)])
    for i, c in enumerate(counts):
        if 0 <= c < T:
            p.k[i, c:] = math.nan
            p.v[i, c:] = math.inf
            p.g[i, c:] = math.nan
    num = torch.tensor(counts, dtype=torch.int32, device="cuda")
    cv.linear_attn_commit(p.k, p.v, p.g, p.pool, num, slot_idx=p.slot_idx)
    torch.cuda.synchronize()
    p.check(want, outputs=False, live=live)
    for i in live:
        if counts[i] == 0:
            assert torch.equal(p.pool_full[p.slots[i].long()].cpu(), p.before[p.slots[i].long()])


@pytest.mark.parametrize("name", ["linear_attn_update", "linear_attn_verify"])
@pytest.mark.parametrize("T", [12, 23, 32])
def test_a_chunk_of_few_tokens_with_strong_decays_and_not_finite(T, name):
    _say("chunk extreme", T, name)
    import causal_conv1d_verify_amd as cv

    p = Problem([T] * 3, 1, 2, 64, 72, "f32", packed=False, T=T, pads=(2,))
    g = p.g.cpu()
    g[0, 4] = -math.inf
    g[1, 2] = -500.0
    p.g = g.cuda()
    want = p.expected()
    p.v[1, 9] = math.nan
    getattr(cv, name)(p.q, p.k, p.v, p.g, p.pool, p.out, slot_idx=p.slot_idx)
    torch.cuda.synchronize()
    got = p.out.cpu()
    for i, upto in ((0, T), (1, 9)):
        a = ref.bounds(want[0][i, :upto], want[2][i, :upto], p.xt, p.xt, p.dk, p.T)
        ref.check(got[i, :upto], want[0][i, :upto], a, f"row {i}")
    assert not torch.isfinite(got[1, 9:]).any()
    slots = [int(s) for s in p.slots]
    if name == "linear_attn_verify":
        assert torch.equal(p.pool_full.cpu(), p.before)
    else:
        a = ref.bounds(want[1][0], want[3][0], p.st, p.xt, p.dk, p.T)
        ref.check(p.pool[slots[0]].cpu(), want[1][0], a, "state")
