"""GPU tests of decayed linear attention (prompts, single tokens, verify and commit) against
the 64-bit recurrence of linear_reference.py, whose bounds are derived there.

Every problem lays q, k and v out as views of one wider buffer (as the conv leaves them), out
with gaps between its heads, the pool with a padded slot stride and unused slots, all filled
with a poison; whatever a call must not write has to keep its bits.
"""

import math

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PAIRS = {"f32": (F32, F32), "bf16": (BF16, BF16), "bf16_f32": (BF16, F32)}
POISON = 7.25


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import causal_conv1d_verify_amd._linattn as L

    L.load()


def _say(*a):
    print("[case]", *a, flush=True)


class Problem:
    """Rows of `lengths` tokens; packed for a prefill, padded to T otherwise."""

    def __init__(self, lengths, hq, hv, dk, dv, pair, *, packed, T=None, decay="token", pads=(),
                 started=None, seed=1, gap=8):
        gen = ref.spread(sum(lengths) + hq * dk, seed)
        self.lengths, self.packed = list(lengths), packed
        n = len(lengths)
        self.T = T = max(1, max(lengths, default=0)) if T is None else T
        self.n, self.hq, self.hv, self.dk, self.dv = n, hq, hv, dk, dv
        self.xt, self.st = PAIRS[pair]
        tokens = sum(lengths) if packed else n * T
        wide = 2 * hq * dk + hv * dv + gap
        buf = torch.randn(tokens, wide, generator=gen)
        self.buf = buf.to(self.xt).cuda()
        self.q = self.buf[:, :hq * dk].unflatten(1, (hq, dk))
        self.k = self.buf[:, hq * dk:2 * hq * dk].unflatten(1, (hq, dk))
        self.v = self.buf[:, 2 * hq * dk:2 * hq * dk + hv * dv].unflatten(1, (hv, dv))
        self.g = {"token": lambda: ref.log_decays((tokens, hv), gen),
                  "head": lambda: ref.log_decays((1, hv), gen)[0] * 0.1,
                  "none": lambda: None}[decay]()
        if self.g is not None:
            self.g = self.g.cuda()
        self.out_full = torch.full((tokens, hv, dv + gap), POISON, dtype=self.xt, device="cuda")
        self.out = self.out_full[..., :dv]
        if not packed:
            self.q, self.k, self.v, self.out = (
                t.unflatten(0, (n, T)) for t in (self.q, self.k, self.v, self.out))
            if decay == "token":
                self.g = self.g.unflatten(0, (n, T))
        self.slots = torch.randperm(n + 3, generator=gen)[:n].to(torch.int32)
        for i in pads:
            self.slots[i] = -1
        area = hv * dk * dv
        self.pool_full = torch.randn(n + 3, area + gap, generator=gen).to(self.st).cuda()
        self.pool = self.pool_full[:, :area].unflatten(1, (hv, dk, dv))
        self.before = self.pool_full.cpu()
        self.slot_idx = self.slots.cuda()
        self.started = None if started is None else torch.tensor(started, dtype=torch.int32)
        starts = [0]
        for t in self.lengths:
            starts.append(starts[-1] + t)
        self.starts = starts
        self.cu = torch.tensor(starts, dtype=torch.int32, device="cuda")

    # -- the recurrence in 64 bits over padded rows --
    def rows(self, t, fill=0.0):
        t = t.cpu()
        if not self.packed:
            return t
        out = torch.full((self.n, self.T, *t.shape[1:]), fill, dtype=t.dtype)
        for i, length in enumerate(self.lengths):
            out[i, :length] = t[self.starts[i]:self.starts[i] + length]
        return out

    def expected(self, counts=None, scale=None):
        if self.g is None:
            g = torch.zeros(self.n, self.T, self.hv)
        elif self.g.dim() == 1:
            g = self.g.cpu().expand(self.n, self.T, self.hv)
        else:
            g = self.rows(self.g)
        area = self.hv * self.dk * self.dv
        first = torch.zeros(self.n, self.hv, self.dk, self.dv, dtype=self.st)
        for i in range(self.n):
            if self.slots[i] >= 0 and (self.started is None or self.started[i]):
                first[i] = self.before[self.slots[i].long(), :area].view(self.hv, self.dk, self.dv)
        return ref.recurrence(self.rows(self.q), self.rows(self.k), self.rows(self.v), g, first,
                              ref.scale_of(self.dk) if scale is None else scale,
                              self.lengths if counts is None else counts)

    def check(self, want, *, outputs=True, state=True, live=None, upto=None):
        """Outputs of live rows, states of their slots; everything else keeps its bits."""
        out, last, out_mass, last_mass = want
        live = [i for i in range(self.n) if self.slots[i] >= 0] if live is None else live
        got = self.out_full.cpu()
        touched = torch.zeros(got.shape[0], dtype=torch.bool)
        worst = [0.0, 0.0]
        for i in live:
            length = self.lengths[i]
            first = self.starts[i] if self.packed else i * self.T
            if outputs and length:
                upto_i = length if upto is None else min(length, upto)
                a = ref.bounds(out[i, :upto_i], out_mass[i, :upto_i], self.xt, self.xt, self.dk, self.T)
                worst[0] = max(worst[0], ref.check(got[first:first + upto_i, :, :self.dv],
                                                   out[i, :upto_i], a, f"out of row {i}"))
                touched[first:first + length] = True
        assert (got[..., self.dv:] == POISON).all(), "gaps of out written"
        assert (got[~touched] == POISON).all(), "rows of out written that must not be"
        pool, area = self.pool_full.cpu(), self.hv * self.dk * self.dv
        kept = torch.ones(pool.shape[0], dtype=torch.bool)
        for i in live:
            if not state:
                break
            slot = int(self.slots[i])
            kept[slot] = False
            a = ref.bounds(last[i], last_mass[i], self.st, self.xt, self.dk, self.T)
            worst[1] = max(worst[1], ref.check(pool[slot, :area].view(self.hv, self.dk, self.dv),
                                               last[i], a, f"state of row {i}"))
        assert torch.equal(pool[kept], self.before[kept]), "untouched slots written"
        assert torch.equal(pool[:, area:], self.before[:, area:]), "pool padding written"
        _say("shares of the bounds: out %.3f, state %.3f" % tuple(worst))

    def prefill(self, **kw):
        import causal_conv1d_verify_amd as cv

        cv.linear_attn_prefill(self.q, self.k, self.v, self.g, self.pool, self.out, self.cu,
                               max_len=self.T, slot_idx=self.slot_idx, has_initial_state=None
                               if self.started is None else self.started.cuda(), **kw)
        torch.cuda.synchronize()


# ---- prompts -------------------------------------------------------------------------

PREFILL = [
    # lengths, hq, hv, dk, dv
    ([1], 1, 1, 8, 8),
    ([2, 0, 31, 32, 33], 1, 2, 16, 24),
    ([63, 64, 65, 1, 0, 128, 129], 2, 4, 64, 64),
    ([100, 3, 190], 1, 3, 128, 128),
    ([70, 200], 2, 2, 96, 72),
    ([140, 64], 1, 1, 256, 256),
    ([67, 66], 1, 2, 200, 136),
    ([90], 3, 3, 40, 248),
    ([700, 5, 1100], 1, 2, 64, 32),
    ([2100, 1], 1, 1, 128, 64),
]


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("shape", PREFILL, ids=lambda s: "-".join(map(str, s[1:])) + f"-L{max(s[0])}")
def test_prefill(shape, pair):
    lengths, hq, hv, dk, dv = shape
    _say("prefill", shape, pair)
    started = [(i + 1) % 2 for i in range(len(lengths))]
    p = Problem(lengths, hq, hv, dk, dv, pair, packed=True, started=started)
    want = p.expected()
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("decay", ["head", "none"])
@pytest.mark.parametrize("pair", PAIRS)
def test_prefill_constant_and_absent_decay(pair, decay):
    _say("prefill decay", pair, decay)
    p = Problem([130, 20, 0, 64], 2, 6, 64, 72, pair, packed=True, decay=decay, pads=(1,))
    want = p.expected()
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("pair", PAIRS)
def test_prefill_many_segments(pair):
    """Rows long enough that their tokens are spread over several workgroups, beside short,
    empty and padded ones; from a state and from zeros."""
    _say("prefill segments", pair)
    p = Problem([4000, 10, 0, 1030, 512, 2049], 1, 2, 64, 64, pair, packed=True, pads=(4,),
                started=[1, 1, 0, 0, 1, 1])
    want = p.expected()
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("pair", PAIRS)
def test_prefill_strong_decays(pair):
    """Decays from none at all to ones that empty the state (-inf among them) next to each
    other: what is left of neighbouring tokens must not lose precision beside them."""
    _say("prefill strong decays", pair)
    p = Problem([300, 65], 1, 2, 64, 32, pair, packed=True)
    g = p.g.cpu()
    g[5::37] = -math.inf
    g[11::41] = -1000.0
    g[17::43] = -1e30
    g[20::5] = 0.0
    p.g = g.cuda()
    want = p.expected()
    p.prefill()
    p.check(want)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("pair", ["f32", "bf16_f32"])
def test_prefill_later_tokens_stay_out(pair, where, bad):
    """A token that is not finite changes its own and later outputs of its row only: not the
    tokens before it, not its packed neighbours."""
    _say("prefill not finite", pair, where, bad)
    p = Problem([100, 150, 90], 1, 2, 64, 32, pair, packed=True)
    want = p.expected()
    at = 77                                      # in row 1, inside a chunk
    getattr(p, where)[p.starts[1] + at] = bad
    p.prefill()
    got = p.out.cpu()
    for i, upto in ((0, 100), (1, at), (2, 90)):
        a = ref.bounds(want[0][i, :upto], want[2][i, :upto], p.xt, p.xt, p.dk, p.T)
        ref.check(got[p.starts[i]:p.starts[i] + upto], want[0][i, :upto], a, f"row {i}")
    after = got[p.starts[1] + at:p.starts[1] + 150]
    if where == "q":                             # its own output alone
        assert not torch.isfinite(after[0]).any()
        a = ref.bounds(want[0][1, at + 1:150], want[2][1, at + 1:150], p.xt, p.xt, p.dk, p.T)
        ref.check(after[1:], want[0][1, at + 1:150], a, "tokens behind")
    else:
        assert not torch.isfinite(after).any()
    pool = p.pool.cpu()
    for i in (0, 2):
        a = ref.bounds(want[1][i], want[3][i], p.st, p.xt, p.dk, p.T)
        ref.check(pool[p.slots[i].long()], want[1][i], a, f"state {i}")


@pytest.mark.parametrize("pair", ["f32", "bf16"])
def test_prefill_bad_rows_are_skipped(pair):
    """Slots outside the pool, a row longer than max_len and falling offsets: nothing of such
    rows is written, the others are right."""
    _say("prefill bad rows", pair)
    p = Problem([70, 20, 33, 90, 12], 1, 2, 32, 40, pair, packed=True)
    want = p.expected()
    p.slot_idx[1] = p.n + 3
    p.slot_idx[2] = -5
    p.T = 80                                     # max_len: row 3 holds 90
    p.prefill()
    p.T = 90
    p.check(want, live=[0, 4])


def test_prefill_falling_offsets():
    _say("prefill falling offsets")
    p = Problem([40, 30], 1, 1, 32, 32, "bf16", packed=True)
    want = p.expected()
    p.cu = torch.tensor([0, 40, 10], dtype=torch.int32, device="cuda")
    p.prefill()
    p.check(want, live=[0])


def test_prefill_is_the_same_every_time():
    _say("prefill repeats")
    p = Problem([1500, 200], 2, 4, 128, 128, "bf16_f32", packed=True)
    p.prefill()
    first = p.out_full.clone(), p.pool_full.clone()
    for _ in range(3):
        p.pool_full.copy_(p.before)
        p.prefill()
        assert torch.equal(first[0], p.out_full) and torch.equal(first[1], p.pool_full)


def test_prefill_in_pieces():
    """A prompt in two calls (the second from the first one's state) gives what one call gives."""
    _say("prefill in pieces")
    p = Problem([500], 1, 2, 64, 64, "bf16_f32", packed=True)
    want = p.expected()
    import causal_conv1d_verify_amd as cv

    for a, b in ((0, 201), (201, 500)):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        cv.linear_attn_prefill(p.q[a:b], p.k[a:b], p.v[a:b], p.g[a:b], p.pool, p.out[a:b], cu,
                               max_len=b - a, slot_idx=p.slot_idx)
    torch.cuda.synchronize()
    p.check(want)


# ---- few tokens ----------------------------------------------------------------------

FEW = [
    # rows, T, hq, hv, dk, dv
    (1, 1, 1, 1, 8, 8),
    (1, 1, 2, 6, 128, 128),
    (5, 1, 1, 3, 96, 72),
    (3, 2, 1, 1, 64, 64),
    (4, 3, 2, 2, 24, 200),
    (3, 8, 2, 4, 128, 128),
    (2, 15, 1, 2, 136, 40),
    (3, 16, 1, 1, 256, 256),
    (4, 17, 1, 3, 64, 128),
    (2, 31, 3, 3, 40, 96),
    (2, 32, 1, 2, 200, 248),
    (300, 1, 1, 2, 64, 64),
    (200, 5, 1, 2, 64, 136),
]


def _few(shape, pair, **kw):
    n, T, hq, hv, dk, dv = shape
    return Problem([T] * n, hq, hv, dk, dv, pair, packed=False, T=T, **kw)


def _call(p, name, *rest, **kw):
    import causal_conv1d_verify_amd as cv

    args = (p.k, p.v, p.g, p.pool) if name == "linear_attn_commit" else \
        (p.q, p.k, p.v, p.g, p.pool, p.out)
    getattr(cv, name)(*args, *rest, slot_idx=p.slot_idx, **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("shape", FEW, ids=lambda s: "-".join(map(str, s)))
def test_update(shape, pair):
    _say("update", shape, pair)
    p = _few(shape, pair, pads=(1,) if shape[0] > 2 else ())
    want = p.expected()
    _call(p, "linear_attn_update")
    p.check(want)


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("shape", FEW, ids=lambda s: "-".join(map(str, s)))
def test_verify_then_commit(shape, pair):
    _say("verify and commit", shape, pair)
    p = _few(shape, pair, pads=(0,) if shape[0] > 2 else ())
    p_out = p.expected()
    _call(p, "linear_attn_verify")
    p.check(p_out, state=False)
    T = shape[1]
    counts = [(5 * i + T) % (T + 1) for i in range(p.n)]
    want = p.expected(counts=counts)
    num = torch.tensor(counts, dtype=torch.int32, device="cuda")
    _call(p, "linear_attn_commit", num)
    p.check((p_out[0], want[1], p_out[2], want[3]))
    for i in range(p.n):                         # nothing accepted: the same bits
        if counts[i] == 0 and p.slots[i] >= 0:
            assert torch.equal(p.pool_full[p.slots[i].long()].cpu(), p.before[p.slots[i].long()])


@pytest.mark.parametrize("decay", ["head", "none"])
@pytest.mark.parametrize("T", [1, 9])
def test_few_tokens_other_decays_and_scale(T, decay):
    _say("few tokens", T, decay)
    p = _few((3, T, 1, 2, 64, 64), "bf16_f32", decay=decay)
    want = p.expected(scale=-1.75)
    _call(p, "linear_attn_update", scale=-1.75)
    p.check(want)


@pytest.mark.parametrize("pair", PAIRS)
def test_commit_of_all_tokens_and_of_bad_counts(pair):
    _say("commit counts", pair)
    p = _few((4, 6, 1, 2, 64, 48), pair)
    want = p.expected(counts=[6, 0, 6, 3])
    num = torch.tensor([6, -1, 7, 3], dtype=torch.int32, device="cuda")
    _call(p, "linear_attn_commit", num)
    p.check(want, outputs=False, live=[0, 3])
    p.pool_full.copy_(p.before)
    _call(p, "linear_attn_commit")
    p.check(p.expected(), outputs=False)


@pytest.mark.parametrize("name", ["linear_attn_update", "linear_attn_verify"])
def test_few_tokens_strong_decays_and_not_finite(name):
    """A draft that is not finite leaves the outputs before it alone; -inf empties the state."""
    _say("few tokens extreme", name)
    p = _few((2, 12, 1, 2, 64, 64), "bf16_f32")
    g = p.g.cpu()
    g[0, 4] = -math.inf
    g[1, 2] = -500.0
    p.g = g.cuda()
    want = p.expected()
    p.v[1, 9] = math.nan
    _call(p, name)
    got = p.out.cpu()
    for i, upto in ((0, 12), (1, 9)):
        a = ref.bounds(want[0][i, :upto], want[2][i, :upto], p.xt, p.xt, p.dk, p.T)
        ref.check(got[i, :upto], want[0][i, :upto], a, f"row {i}")
    assert not torch.isfinite(got[1, 9:]).any()


@pytest.mark.parametrize("T", [1, 6])
def test_commit_does_not_read_rejected_tokens(T):
    _say("commit rejected", T)
    p = _few((2, T + 2, 1, 1, 64, 64), "bf16_f32")
    want = p.expected(counts=[T, T])
    p.k[:, T:] = math.nan
    p.v[:, T:] = math.inf
    p.g[:, T:] = math.nan
    _call(p, "linear_attn_commit", torch.full((2,), T, dtype=torch.int32, device="cuda"))
    p.check(want, outputs=False)


def test_token_by_token_is_the_prompt():
    """Single tokens one after the other reach the state and outputs of the prompt."""
    _say("tokens against prompt")
    p = _few((2, 40, 1, 2, 64, 64), "bf16_f32")
    want = p.expected()
    import causal_conv1d_verify_amd as cv

    for t in range(40):
        cv.linear_attn_update(p.q[:, t:t + 1], p.k[:, t:t + 1], p.v[:, t:t + 1], p.g[:, t:t + 1],
                              p.pool, p.out[:, t:t + 1], slot_idx=p.slot_idx)
    torch.cuda.synchronize()
    p.check(want)


# ---- layouts, offsets, streams, graphs -----------------------------------------------


@pytest.mark.parametrize("T", [1, 7])
def test_heads_before_tokens(T):
    """[n, heads, T, channels] storage seen as [n, T, heads, channels]; broadcast k."""
    _say("heads before tokens", T)
    import causal_conv1d_verify_amd as cv

    gen = ref.spread(T, 5)
    n, hq, hv, dk, dv = 2, 2, 4, 64, 32
    q = torch.randn(n, hq, T, dk, generator=gen).to(BF16).cuda().transpose(1, 2)
    k = torch.randn(n, T, 1, dk, generator=gen).to(BF16).cuda().expand(n, T, hq, dk)
    v = torch.randn(n, hv, T, dv, generator=gen).to(BF16).cuda().transpose(1, 2)
    out = torch.full((n, hv, T, dv), POISON, dtype=BF16, device="cuda").transpose(1, 2)
    g = ref.log_decays((n, T, hv), gen)
    pool = torch.randn(n, hv, dk, dv, generator=gen)
    want = ref.recurrence(q.cpu(), k.cpu(), v.cpu(), g, pool, ref.scale_of(dk))
    pool = pool.cuda()
    cv.linear_attn_update(q, k, v, g.cuda(), pool, out)
    torch.cuda.synchronize()
    ref.check(out, want[0], ref.bounds(want[0], want[2], BF16, BF16, dk, T), "out")
    ref.check(pool, want[1], ref.bounds(want[1], want[3], F32, BF16, dk, T), "state")


def test_offsets_past_32_bits():
    """Slots, tokens and rows further than 2^31 elements (2^32 bytes) from their pointers."""
    _say("offsets")
    import causal_conv1d_verify_amd as cv

    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    gen = ref.spread(3, 9)
    d, T, far = 32, 70, 1 << 25                # 70 tokens 2^25 elements apart: 2.3e9 elements
    wide = torch.empty(T * far, dtype=BF16, device="cuda")
    qkv = wide.as_strided((T, 3, d), (far, d, 1))
    host = torch.randn(T, 3, d, generator=gen).to(BF16)
    qkv.copy_(host)
    out = wide.as_strided((T, 1, d), (far, d, 1), 4096)
    pools = torch.empty((1 << 31) + 4096, dtype=BF16, device="cuda")
    pool = pools.as_strided((2, 1, d, d), (1 << 31, d * d, d, 1))
    pool.copy_(torch.randn(2, 1, d, d, generator=gen))
    before = pool.cpu()
    g = ref.log_decays((T, 1), gen)
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    want = ref.recurrence(host[None, :, 0:1], host[None, :, 1:2], host[None, :, 2:3], g[None],
                          before[1:2], ref.scale_of(d))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    cv.linear_attn_prefill(qkv[:, 0:1], qkv[:, 1:2], qkv[:, 2:3], g.cuda(), pool, out, cu,
                           max_len=T, slot_idx=slot)
    torch.cuda.synchronize()
    ref.check(out.cpu()[None], want[0], ref.bounds(want[0], want[2], BF16, BF16, d, T), "out")
    ref.check(pool[1:2].cpu(), want[1], ref.bounds(want[1], want[3], BF16, BF16, d, T), "state")
    assert torch.equal(pool[0].cpu(), before[0])
    # 8 single-token rows, each 2^28 elements apart, on the far slot's neighbours
    pool.copy_(before)
    rows = wide.as_strided((2, 8, 3, d), (1 << 30, far, d, 1))
    want = ref.recurrence(rows[:, :, 0:1].cpu(), rows[:, :, 1:2].cpu(), rows[:, :, 2:3].cpu(),
                          torch.zeros(2, 8, 1), before, ref.scale_of(d))
    res = wide.as_strided((2, 8, 1, d), (1 << 30, far, d, 1), 8192)
    cv.linear_attn_update(rows[:, :, 0:1], rows[:, :, 1:2], rows[:, :, 2:3], None, pool, res)
    torch.cuda.synchronize()
    ref.check(res.cpu(), want[0], ref.bounds(want[0], want[2], BF16, BF16, d, 8), "out")
    ref.check(pool.cpu(), want[1], ref.bounds(want[1], want[3], BF16, BF16, d, 8), "state")


def test_on_another_stream():
    """On a stream that is not torch's current one, with the workspace made by the call."""
    _say("stream")
    p = Problem([2000, 300], 1, 2, 64, 64, "bf16_f32", packed=True)
    want = p.expected()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.prefill(stream=s)
    s.synchronize()
    p.check(want)
    q = _few((3, 5, 1, 2, 64, 64), "bf16_f32")
    s.wait_stream(torch.cuda.current_stream())
    want = q.expected()
    _call(q, "linear_attn_update", stream=s)
    s.synchronize()
    q.check(want)


def test_graph_replays():
    """A captured step (prompt, verify, commit, single token, the norms), replayed with eager
    work between the replays, gives the bits of the eager step every time."""
    _say("graph")
    import causal_conv1d_verify_amd as cv

    p = Problem([1300, 40], 1, 2, 64, 64, "bf16_f32", packed=True)
    f = _few((2, 6, 1, 2, 64, 64), "bf16_f32", seed=2)
    f.pool, f.slot_idx = p.pool, p.slot_idx
    num = torch.tensor([4, 6], dtype=torch.int32, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    normed = torch.zeros(2, 6, 2, 64, dtype=BF16, device="cuda")
    res = torch.zeros(12, 128, dtype=BF16, device="cuda")
    nxt = torch.zeros_like(res)
    w2 = torch.ones(128, dtype=BF16, device="cuda")

    def step():
        cv.linear_attn_prefill(p.q, p.k, p.v, p.g, p.pool, p.out, p.cu, max_len=p.T,
                               slot_idx=p.slot_idx)
        cv.linear_attn_verify(f.q, f.k, f.v, f.g, f.pool, f.out, slot_idx=f.slot_idx)
        cv.linear_attn_commit(f.k, f.v, f.g, f.pool, num, slot_idx=f.slot_idx)
        cv.linear_attn_update(f.q[:, :1], f.k[:, :1], f.v[:, :1], f.g[:, :1], f.pool,
                              f.out[:, :1], slot_idx=f.slot_idx)
        cv.gated_norm(f.out.flatten(0, 1), f.v.flatten(0, 1), w, normed.flatten(0, 1))
        cv.residual_norm(normed.view(12, 128), res, w2, nxt, post_weight=w2)

    def fresh():
        p.pool_full.copy_(p.before)
        p.out_full.fill_(POISON)
        f.out_full.fill_(POISON)
        res.fill_(0.5)
        nxt.zero_()

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (p.pool_full, p.out_full, f.out_full, normed, res, nxt)]

    fresh()
    step()
    eager = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        fresh()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), eager))
        fresh()
        step()
        assert all(torch.equal(a, b) for a, b in zip(results(), eager))


def test_nothing_to_do():
    _say("empty")
    p = Problem([0, 0], 1, 2, 64, 64, "bf16_f32", packed=True, started=[1, 0])
    want = p.expected()
    p.prefill()
    p.check(want)                                # one state kept, one emptied
    import causal_conv1d_verify_amd as cv

    none = p.q.new_empty(0, 3, 1, 64)
    cv.linear_attn_update(none, none, none, None, p.pool[:, :1], none)
    torch.cuda.synchronize()
