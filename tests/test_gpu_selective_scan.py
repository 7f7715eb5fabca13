"""GPU tests of the selective scan (prompts, single tokens, verify and commit) against the 64-bit
recurrence of sequence_reference.py, whose bounds are derived there.

Every problem lays z out in a wider buffer, B and C in another at odd offsets, out with gaps between
its rows, the pool with a padded slot stride and unused slots, all filled with a poison; whatever a
call must not write has to keep its bits.
"""

import pytest
import torch

import sequence_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PAIRS = {"f32": (F32, F32), "bf16": (BF16, BF16), "bf16_f32": (BF16, F32)}
POISON = 7.25


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from causal_conv1d_verify_amd import _seqops

    _seqops.load()


def _say(*a):
    print("[case]", *a, flush=True)


def rand(*shape, gen):
    return torch.randn(*shape, generator=gen)


class Problem:
    """Rows of `lengths` tokens; packed for a prefill, of T tokens each otherwise."""

    def __init__(self, lengths, d, n, pair, *, packed, T=None, gate=True, skip=True, bias=True,
                 softplus=True, pads=(), started=None, seed=1, off=1):
        gen = torch.Generator().manual_seed(seed)
        self.lengths, self.packed, self.d, self.n = list(lengths), packed, d, n
        rows = self.rows = len(lengths)
        self.T = T = max(1, max(lengths, default=0)) if T is None else T
        self.xt, self.st = PAIRS[pair]
        tokens = sum(lengths) if packed else rows * T
        self.tokens = tokens

        def put(t, dtype=None):
            return t.to(self.xt if dtype is None else dtype).cuda()

        self.x = put(rand(tokens, d, gen=gen))
        raw = rand(tokens, d, gen=gen) - (0 if bias else 3)
        self.dt = put(raw if softplus else 0.3 * torch.rand(tokens, d, generator=gen))
        self.z = put(rand(tokens, 2 * d + 16, gen=gen))[:, d + 16:] if gate else None
        # B and C at an offset that no vector is aligned to
        low = put(rand(tokens, off + 2 * n + 3, gen=gen))
        self.B, self.C = low[:, off:off + n], low[:, off + n:off + 2 * n]
        self.A = -(torch.arange(1, n + 1) * (0.5 + torch.rand(d, n, generator=gen))).float().cuda()
        self.D = rand(d, gen=gen).cuda() if skip else None
        self.dt_bias = (rand(d, gen=gen) - 3).cuda() if bias else None
        self.softplus = softplus
        self.out_full = torch.full((tokens, d + 16), POISON, dtype=self.xt, device="cuda")
        self.out = self.out_full[:, :d]
        slots = torch.randperm(rows + 2, generator=gen)[:rows].to(torch.int32)
        for i in pads:
            slots[i] = -1
        self.slots = slots.cuda()
        self.pool_full = put(rand(rows + 2, d * n + 16, gen=gen), self.st)
        self.pool = self.pool_full[:, :d * n].unflatten(1, (d, n))
        self.cu = torch.tensor([0, *torch.tensor(self.lengths).cumsum(0).tolist()], dtype=torch.int32).cuda()
        self.started = None if started is None else torch.tensor(started, dtype=torch.int32).cuda()
        if not packed:
            for name in ("x", "dt", "z", "B", "C", "out"):
                t = getattr(self, name)
                setattr(self, name, None if t is None else t.unflatten(0, (rows, T)))

    def kw(self, out=True, **more):
        kw = dict(dt_bias=self.dt_bias, dt_softplus=self.softplus, slot_idx=self.slots, **more)
        return dict(kw, z=self.z, D=self.D) if out else kw

    def row(self, i):
        """Row i's token tensors, [L, ...] on the CPU."""
        if self.packed:
            at = slice(int(self.cu[i]), int(self.cu[i]) + self.lengths[i])
            return [None if t is None else t[at].cpu() for t in (self.x, self.dt, self.B, self.C, self.z)]
        return [None if t is None else t[i].cpu() for t in (self.x, self.dt, self.B, self.C, self.z)]

    def expect(self, taken=None, outputs=True, writes=True):
        """What out and the pool must hold and how far off they may be (0: the same bits)."""
        out, pool = self.out_full.cpu().double(), self.pool_full.cpu().double()
        out_tol, pool_tol = torch.zeros_like(out), torch.zeros_like(pool)
        slots, A = self.slots.cpu(), self.A.cpu()
        D, bias = (None if t is None else t.cpu() for t in (self.D, self.dt_bias))
        d, n = self.d, self.n
        for i in range(self.rows):
            s = int(slots[i])
            if s < 0:
                continue
            x, dt, B, C, z = self.row(i)
            L = x.shape[0] if self.packed else self.T
            first = pool[s, :d * n].view(d, n)
            fresh = self.started is not None and not int(self.started[i])
            row = ref.Scan(torch.zeros_like(first) if fresh else first, A, D, bias, self.softplus)
            base = int(self.cu[i]) if self.packed else i * self.T
            count = L if taken is None else int(taken[i])
            if not 0 <= count <= L:
                continue
            state = row.state()
            for t in range(L):
                if outputs:
                    y, tol = row.token(x[t], dt[t], B[t], C[t], None if z is None else z[t])
                    out[base + t, :d], out_tol[base + t, :d] = y, ref.rounded(y, tol, self.xt)
                elif t < count:
                    row.token(x[t], dt[t], B[t])
                if t + 1 == count:
                    state = row.state()
            if writes and (count or fresh):
                h, tol = state
                pool[s, :d * n], pool_tol[s, :d * n] = h.flatten(), ref.rounded(h, tol, self.st).flatten()
        return out, out_tol, pool, pool_tol

    def check(self, want):
        torch.cuda.synchronize()
        out, out_tol, pool, pool_tol = want
        for name, got, exp, tol in (("out", self.out_full, out, out_tol), ("pool", self.pool_full, pool, pool_tol)):
            off = (got.cpu().double() - exp).abs()
            bad = ~(off <= tol) & torch.isfinite(tol)
            assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4].tolist(),
                                   off[bad][:4].tolist(), tol[bad][:4].tolist())


def _cv():
    import causal_conv1d_verify_amd as cv

    return cv


def prefill(p, **more):
    _cv().selective_scan_prefill(p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, p.cu, max_len=p.T,
                                 has_initial_state=p.started, **p.kw(**more))


ROWS = {"one": [1], "ragged": [5, 0, 33, 1, 16, 4], "stage": [15, 16, 17, 31, 32], "long": [300, 2, 129]}


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d,n", [(8, 8), (64, 16), (104, 16), (72, 24), (136, 32), (48, 40), (64, 48), (24, 56),
                                 (40, 64)])
def test_prompts(pair, rows, d, n):
    _say(pair, rows, d, n)
    lengths = ROWS[rows]
    started = [i % 3 != 1 for i in range(len(lengths))]
    p = Problem(lengths, d, n, pair, packed=True, started=started, pads=(3,) if len(lengths) > 4 else (), seed=d + n)
    want = p.expect()
    prefill(p)
    p.check(want)


@pytest.mark.parametrize("gate,skip,bias,softplus", [(False, False, False, True), (True, False, False, False),
                                                     (False, True, True, False), (False, False, True, True)])
def test_prompts_without_some(gate, skip, bias, softplus):
    _say(gate, skip, bias, softplus)
    p = Problem([20, 3, 50], 72, 16, "bf16_f32", packed=True, gate=gate, skip=skip, bias=bias, softplus=softplus)
    want = p.expect()
    prefill(p)
    p.check(want)


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("lengths,d,n,started", [
    ([1000], 64, 16, [1]), ([1000], 72, 16, [0]), ([700, 3, 0, 655], 128, 8, [1, 0, 0, 1]),
    ([2, 1500, 64, 65], 40, 24, [1, 0, 1, 1]), ([129, 1030], 24, 64, [0, 1])])
def test_prompts_that_are_cut(pair, lengths, d, n, started):
    """Rows in segments, whose states are joined; the description says that they are."""
    _say(pair, lengths, d, n)
    p = Problem(lengths, d, n, pair, packed=True, started=started, seed=len(lengths))
    info = _cv().selective_scan_describe("prefill", p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, p.cu, max_len=p.T,
                                         has_initial_state=p.started, **p.kw())
    assert info.launches == 2 and 0 < info.segment_tokens < max(lengths)
    want = p.expect()
    prefill(p)
    p.check(want)


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("T", [1, 2, 4, 5, 15, 16, 17, 32])
@pytest.mark.parametrize("d,n", [(64, 16), (200, 16), (16, 8), (72, 24), (24, 64)])
def test_update_verify_commit(pair, T, d, n):
    _say(pair, T, d, n)
    cv = _cv()
    for kind in ("update", "verify", "commit"):
        p = Problem([T] * 5, d, n, pair, packed=False, T=T, pads=(2,), seed=T + d)
        if kind == "commit":
            num = torch.tensor([0, T, T, (T + 1) // 2, T + 1], dtype=torch.int32)   # the last: out of range
            want = p.expect(taken=num, outputs=False)
            cv.selective_scan_commit(p.x, p.dt, p.A, p.B, p.pool, num.cuda(), **p.kw(out=False))
        else:
            want = p.expect(writes=kind == "update")
            getattr(cv, "selective_scan_" + kind)(p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, **p.kw())
        p.check(want)


def test_commit_of_all_tokens_and_no_slots():
    _say("commit all")
    p = Problem([6] * 3, 80, 16, "bf16_f32", packed=False, T=6)
    p.slots = torch.arange(3, dtype=torch.int32).cuda()
    want = p.expect(outputs=False)
    _cv().selective_scan_commit(p.x, p.dt, p.A, p.B, p.pool, dt_bias=p.dt_bias)
    p.check(want)


@pytest.mark.parametrize("lengths", [[], [0], [0, 0, 0]], ids=str)
@pytest.mark.parametrize("fresh", [False, True])
def test_prompts_without_tokens(lengths, fresh):
    """States stay as they are, or start from zeros."""
    _say(lengths, fresh)
    p = Problem(lengths, 64, 16, "f32", packed=True, started=[0] * len(lengths) if fresh else None)
    want = p.expect()
    prefill(p)
    p.check(want)


def test_more_tokens_than_declared():
    """Rows longer than max_len, and slots out of the pool, are skipped."""
    _say("declared")
    p = Problem([9, 40, 7, 5], 64, 16, "bf16", packed=True, T=10)
    p.slots[3] = p.pool.shape[0]
    slots = p.slots.clone()
    p.slots[1] = p.slots[3] = -1
    want = p.expect()
    p.slots = slots
    prefill(p)
    p.check(want)


@pytest.mark.parametrize("where", ["x", "dt", "z", "B", "C"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_values_that_are_not_finite_stay_behind(where, value):
    """Tokens before such a value, other rows and (but for B and C) other channels keep their bits."""
    _say(where, value)
    lengths, token, channel = [90, 40], 50, 9
    clean = Problem(lengths, 72, 16, "bf16_f32", packed=True)
    prefill(clean)
    p = Problem(lengths, 72, 16, "bf16_f32", packed=True)
    getattr(p, where)[token, channel] = value
    prefill(p)
    torch.cuda.synchronize()
    same = torch.ones_like(p.out, dtype=torch.bool)
    if where in ("B", "C"):
        same[token:90 if where == "B" else token + 1] = False
    else:
        same[token:90 if where != "z" else token + 1, channel] = False
    assert torch.equal(p.out[same], clean.out[same])
    assert not torch.isfinite(p.out[token, channel].float())


@pytest.mark.parametrize("dt", [-200.0, -90.0, -30.0, 0.0, 40.0, 1e30])
def test_steps_far_out(dt):
    """Softplus at its ends: no step at all, or a decay that empties the state."""
    _say(dt)
    p = Problem([40], 64, 16, "f32", packed=True, bias=False, gate=False)
    p.dt.fill_(dt)
    if dt == 1e30:
        p.x.zero_()
    want = p.expect()
    prefill(p)
    p.check(want)


def test_a_captured_call_replayed():
    """Segments, verify and commit in one graph, replayed between eager calls."""
    _say("graph")
    cv = _cv()
    p = Problem([900, 3], 72, 16, "bf16_f32", packed=True, started=[0, 0])
    q = Problem([8] * 4, 72, 16, "bf16_f32", packed=False, T=8)
    num = torch.tensor([3, 8, 0, 1], dtype=torch.int32).cuda()
    want, first = p.expect(), q.pool_full.clone()
    verify, commit = q.expect(writes=False), q.expect(taken=num, outputs=False)

    def step():
        prefill(p)
        cv.selective_scan_verify(q.x, q.dt, q.A, q.B, q.C, q.pool, q.out, **q.kw())
        cv.selective_scan_commit(q.x, q.dt, q.A, q.B, q.pool, num, **q.kw(out=False))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        p.out.fill_(POISON), q.out.fill_(POISON)
        q.pool_full.copy_(first)
        graph.replay()
        p.check(want)
        q.check((verify[0], verify[1], commit[2], commit[3]))
        other = Problem([70], 64, 16, "f32", packed=True)
        prefill(other)


def test_another_stream_and_both_ways():
    """The binding's own way (a stream is named) gives the call module's bits."""
    _say("stream")
    a, b = (Problem([900, 40], 72, 16, "bf16_f32", packed=True) for _ in range(2))
    prefill(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    prefill(b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.pool_full, b.pool_full)


def test_prepared_calls():
    _say("prepared")
    cv = _cv()
    p = Problem([4] * 3, 64, 16, "bf16", packed=False, T=4)
    want = p.expect(writes=False)
    launch = cv.prepare("selective_scan_verify", p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, **p.kw())
    launch()
    p.check(want)


def test_rows_past_32_bit_offsets():
    """Token rows 2^28 elements apart: the last ones lie past 4 GiB."""
    _say("far rows")
    p = Problem([9], 64, 16, "bf16_f32", packed=True)
    far = 2 ** 28
    for name in ("x", "dt", "out", "z"):
        wide = torch.empty(8 * far + 64, dtype=BF16, device="cuda")
        view = torch.as_strided(wide, (9, 64), (far, 1))
        view.copy_(getattr(p, name))
        setattr(p, name, view)
    q = Problem([9], 64, 16, "bf16_f32", packed=True)
    prefill(p)
    prefill(q)
    torch.cuda.synchronize()
    assert torch.equal(p.out, q.out) and torch.equal(p.pool_full, q.pool_full)


def test_few_tokens_too_far_apart():
    """Token rows 2^29 elements apart, past the 32-bit offsets of the kernel that takes near ones."""
    _say("few far rows")
    cv = _cv()
    far = 2 ** 29
    for kind in ("verify", "update"):
        p, q = (Problem([9] * 2, 64, 16, "bf16_f32", packed=False, T=9) for _ in range(2))
        wide = torch.empty(8 * far + 2 * 64, dtype=BF16, device="cuda")
        view = torch.as_strided(wide, (2, 9, 64), (64, far, 1))
        view.copy_(p.x)
        p.x = view
        want = q.expect(writes=kind == "update")
        for r in (p, q):
            getattr(cv, "selective_scan_" + kind)(r.x, r.dt, r.A, r.B, r.C, r.pool, r.out, **r.kw())
            r.check(want)


@pytest.mark.parametrize("packed", [True, False])
def test_inputs_that_are_broadcast(packed):
    """One dt, z, B and C for all tokens (stride 0)."""
    _say("broadcast", packed)
    cv = _cv()
    p = Problem([21] * 3, 72, 16, "bf16_f32", packed=packed, T=21)
    for name in ("dt", "z", "B", "C"):
        t = getattr(p, name)
        first = t[:1] if packed else t[:, :1]
        setattr(p, name, first.expand_as(t))
    want = p.expect()
    if packed:
        prefill(p)
    else:
        cv.selective_scan_update(p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, **p.kw())
    p.check(want)


def test_tokens_behind_the_last_row_are_left():
    _say("tail")
    p = Problem([30, 17, 9], 72, 16, "bf16_f32", packed=True)
    p.cu = p.cu[:-1].contiguous()
    p.rows, p.lengths, p.slots = 2, p.lengths[:2], p.slots[:2].contiguous()
    want = p.expect()
    prefill(p)
    p.check(want)


def test_two_calls_at_once():
    """Cut prompts on two streams, each with a workspace of its own."""
    _say("two streams")
    ps = [Problem([1200, 40], 72, 16, "bf16_f32", packed=True, seed=k) for k in range(2)]
    wants = [p.expect() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for p, s in zip(ps, streams):
        with torch.cuda.stream(s):
            prefill(p)
    for p, want in zip(ps, wants):
        p.check(want)


@pytest.mark.parametrize("d,n", [(64, 16), (72, 24), (24, 64)])
def test_rows_of_no_tokens_at_either_end(d, n):
    _say("no tokens at either end", d, n)
    p = Problem([0, 0, 21, 0], d, n, "bf16_f32", packed=True, started=[0, 1, 0, 0])
    want = p.expect()
    prefill(p)
    p.check(want)


@pytest.mark.parametrize("kind,tokens", [("prefill", 1), ("prefill", 5), ("prefill", 18), ("update", 9), ("update", 18)])
@pytest.mark.parametrize("where", ["x", "B"])
def test_an_infinity_in_every_token(kind, tokens, where):
    """x or B is one row for all tokens, with an infinity: a state that it reaches is that infinity, not
    what 0 times it would be for tokens past the row's end."""
    _say("infinity", kind, tokens, where)
    d, n = 64, 16
    row = torch.ones(d if where == "x" else n, device="cuda")
    row[3] = float("inf")
    lead = (tokens,) if kind == "prefill" else (2, tokens)
    x = row.expand(*lead, d) if where == "x" else torch.ones(*lead, d, device="cuda")
    B = row.expand(*lead, n) if where == "B" else torch.ones(*lead, n, device="cuda")
    dt, C = torch.zeros(*lead, d, device="cuda"), torch.ones(*lead, n, device="cuda")
    A = -torch.ones(d, n, device="cuda")
    state, out = torch.ones(2, d, n, device="cuda"), torch.zeros(*lead, d, device="cuda")
    if kind == "prefill":
        cu = torch.tensor([0, tokens], dtype=torch.int32).cuda()
        _cv().selective_scan_prefill(x, dt, A, B, C, state, out, cu, max_len=tokens)
        state, out = state[:1], out[None]
    else:
        _cv().selective_scan_update(x, dt, A, B, C, state, out)
    hit = torch.zeros(d, n, dtype=torch.bool)
    (hit[3] if where == "x" else hit[:, 3]).fill_(True)
    assert torch.equal(torch.isposinf(state).cpu(), hit.expand(state.shape))
    assert torch.isfinite(state.cpu()[~hit.expand(state.shape)]).all()
    assert torch.equal(torch.isposinf(out).cpu(), hit.any(1).expand(out.shape))
    assert torch.isfinite(out.cpu()[~hit.any(1).expand(out.shape)]).all()


@pytest.mark.parametrize("n", [16, 24, 64])
def test_growth_of_nothing(n):
    """A state of zeros stays zeros however much it would have grown (e^4 a token, over segments of 64
    and more), and the last token's values are whole numbers."""
    _say("growth of nothing", n)
    tokens, d = 1024, 64
    x = torch.zeros(tokens, d, device="cuda")
    x[-1] = -2.0
    dt = torch.full((tokens, d), -1.0, device="cuda")
    A = torch.full((d, n), -4.0, device="cuda")
    B, C = torch.ones(tokens, n, device="cuda"), torch.ones(tokens, n, device="cuda")
    state, out = torch.ones(1, d, n, device="cuda"), torch.full((tokens, d), POISON, device="cuda")
    cu = torch.tensor([0, tokens], dtype=torch.int32).cuda()
    kw = dict(max_len=tokens, dt_softplus=False, has_initial_state=torch.zeros(1, dtype=torch.int32).cuda())
    import causal_conv1d_verify_amd.sequence_ops as sq

    assert sq.selective_scan_describe("prefill", x, dt, A, B, C, state, out, cu, **kw).segment_tokens > 0
    _cv().selective_scan_prefill(x, dt, A, B, C, state, out, cu, **kw)
    assert torch.equal(state.cpu(), torch.full((1, d, n), 2.0))
    assert torch.equal(out[:-1].cpu(), torch.zeros(tokens - 1, d))
    assert torch.equal(out[-1].cpu(), torch.full((d,), 2.0 * n))


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("T", [8, 9, 12, 13, 20, 21, 24, 25])
@pytest.mark.parametrize("d,n", [(64, 16), (40, 24), (24, 48), (16, 64)])
def test_few_tokens_in_stages(pair, T, d, n):
    """A group of four tokens more and less than the stages hold."""
    _say("stages", pair, T, d, n)
    for kind, write in (("selective_scan_verify", False), ("selective_scan_update", True)):
        p = Problem([T] * 3, d, n, pair, packed=False, T=T, pads=(1,), seed=T + n)
        want = p.expect(writes=write)
        getattr(_cv(), kind)(p.x, p.dt, p.A, p.B, p.C, p.pool, p.out, **p.kw())
        p.check(want)
