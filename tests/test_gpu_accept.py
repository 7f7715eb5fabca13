"""GPU tests of the verdict on drafts against sequence_reference.verdict: whole numbers, which have to be
equal.  (Sums of fp64 in two orders differ by 2^-53 of themselves a term; a given random number falls
between two of them with a chance of about 1e-10 a row, and the inputs here are fixed.)"""

import pytest
import torch

import sequence_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
POISON = -77


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from causal_conv1d_verify_amd import _seqops

    _seqops.load()


def _cv():
    import causal_conv1d_verify_amd as cv

    return cv


def _say(*a):
    print("[case]", *a, flush=True)


class Problem:
    """CPU tensors of n rows of T tokens over a vocabulary; `kind`: chain (drawn drafts), certain
    (no draft's probabilities) or tree."""

    def __init__(self, n, T, vocab, kind, dtype=F32, *, seed=1, sharp=2.0, near=0.7, pads=()):
        gen = torch.Generator().manual_seed(seed)
        logits = sharp * torch.randn(n, T, vocab, generator=gen)
        self.n, self.T, self.vocab = n, T, vocab
        self.target = logits.softmax(-1).to(dtype)
        self.draft = self.parent = None
        if kind == "chain":
            self.draft = (logits[:, :T - 1] + near * torch.randn(n, T - 1, vocab, generator=gen)).softmax(-1).to(dtype)
            source = self.draft
        elif kind == "tree":
            back = 1 + (torch.rand(n, T, generator=gen) * 4).int()
            self.parent = (torch.arange(T, dtype=torch.int32) - back).clamp(min=0)
            self.parent[:, 0] = -1
            source = self.target.gather(1, self.parent[:, 1:, None].long().expand(-1, -1, vocab))
        else:
            source = self.target[:, :T - 1]
        self.tokens = torch.randint(0, vocab, (n, T), generator=gen, dtype=torch.int32)
        if T > 1:
            p = source.float().flatten(0, 1)
            self.tokens[:, 1:] = torch.multinomial(p, 1, generator=gen).view(n, T - 1).int()
        self.uniform = torch.rand(n, T, generator=gen)
        self.slots = torch.arange(n, dtype=torch.int32)
        for i in pads:
            self.slots[i] = -1

    def expect(self):
        num, nxt, last = (torch.full((self.n,), POISON, dtype=torch.int32) for _ in range(3))
        path = torch.full((self.n, self.T), POISON, dtype=torch.int32)
        for i in range(self.n):
            if self.slots[i] < 0:
                continue
            r = ref.verdict(self.tokens[i], self.target[i], self.uniform[i],
                            None if self.draft is None else self.draft[i],
                            None if self.parent is None else self.parent[i])
            if r is not None:
                num[i], nxt[i], last[i] = r[:3]
                path[i] = torch.tensor(r[3], dtype=torch.int32)
        return num, nxt, last, path

    def gpu(self):
        self.out = [torch.full((self.n,), POISON, dtype=torch.int32, device="cuda") for _ in range(3)]
        self.path = torch.full((self.n, self.T + 3), POISON, dtype=torch.int32, device="cuda")
        # rows of odd lengths apart, so that they start off every vector
        def odd(t):
            if t is None:
                return None
            wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype, device="cuda")
            wide[..., :-1] = t.cuda()
            return wide[..., :-1]

        self.args = [self.tokens.cuda(), odd(self.target), self.uniform.cuda()]
        self.kw = dict(draft=odd(self.draft), parent=None if self.parent is None else self.parent.cuda(),
                       window_index=self.out[2], path=self.path[:, :self.T], slot_idx=self.slots.cuda())

    def call(self, **more):
        _cv().accept_drafts(*self.args, *self.out[:2], **self.kw, **more)

    def check(self, want):
        torch.cuda.synchronize()
        got = [t.cpu() for t in (*self.out, self.path[:, :self.T])]
        for name, g, w in zip(("num_tokens", "next_token", "window_index", "path"), got, want):
            assert torch.equal(g, w), (name, (g != w).nonzero()[:4].tolist(), g[g != w][:4], w[g != w][:4])
        assert bool((self.path[:, self.T:] == POISON).all())

    def run(self):
        want = self.expect()
        self.gpu()
        self.call()
        self.check(want)
        return want


@pytest.mark.parametrize("kind", ["chain", "certain", "tree"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("n,T,vocab", [(1, 1, 1), (1, 1, 5000), (3, 2, 7), (40, 8, 97), (6, 17, 1023), (5, 32, 1025),
                                       (4, 5, 4096), (2, 4, 9999), (1, 3, 70001)])
def test_rows(kind, dtype, n, T, vocab):
    _say(kind, dtype, n, T, vocab)
    Problem(n, T, vocab, kind, dtype, seed=vocab + T).run()


@pytest.mark.parametrize("kind", ["chain", "certain", "tree"])
def test_many_rows(kind):
    """Every verdict occurs: none, some and all of the drafts accepted."""
    _say(kind)
    num = Problem(700, 6, 61, kind, seed=3, near=0.5, sharp=4.0, pads=(5, 600)).run()[0]
    assert {int(x) for x in num} >= ({1, 2, 3} if kind == "tree" else {1, 2, 3, 4, 5, 6}) | {POISON}


@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_pads_among_the_tokens(kind):
    """-1, a token past the vocabulary and the least int32 are not tried; what comes behind one in a
    chain is not reached."""
    _say(kind)
    p = Problem(60, 9, 50, kind, seed=5, sharp=4.0)
    p.tokens[:, 4] = -1
    p.tokens[::2, 2] = 50
    p.tokens[::3, 6] = -2 ** 31
    p.run()


def test_trees_with_unused_tokens_and_with_faults():
    """Parent -1: never reached.  A parent that is not before its child: the row is skipped."""
    _say("parents")
    p = Problem(12, 8, 40, "tree", seed=6)
    p.parent[:, 5:] = -1
    p.parent[1, 3] = 3
    p.parent[2, 1] = -2
    p.parent[3, 0] = 0
    p.parent[4, 7] = 2 ** 31 - 1
    want = p.run()
    assert [int(want[0][i]) for i in (1, 2, 3, 4)] == [POISON] * 4


def test_children_of_the_same_token():
    """The second of two is not accepted, nor does it weigh twice."""
    _say("twins")
    p = Problem(200, 7, 5, "tree", seed=7)
    p.parent[:] = torch.tensor([-1, 0, 0, 0, 0, 0, 0], dtype=torch.int32)
    p.run()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_random_numbers_at_their_ends(dtype):
    _say(dtype)
    for value in (0.0, 1.0 - 2.0 ** -24, 0.5):
        for kind in ("chain", "certain", "tree"):
            p = Problem(20, 5, 300, kind, dtype, seed=8)
            p.uniform.fill_(value)
            p.run()


def _certain(vocab, at):
    p = torch.zeros(vocab)
    p[at] = 1.0
    return p


def test_probabilities_of_zero_and_one():
    """Sharp distributions, ties at borders, a residual of nothing."""
    _say("sharp")
    V = 2500
    p = Problem(6, 3, V, "chain", seed=9)
    p.target[:], p.draft[:] = 0, 0
    for i in range(6):
        p.tokens[i, 1:] = torch.tensor([7, 2400])
        p.draft[i, 0], p.draft[i, 1] = _certain(V, 7), _certain(V, 2400)
        for t in range(3):
            p.target[i, t] = _certain(V, (7, 2400, 2499)[t])
    p.target[1, 0] = _certain(V, 8)          # rejected at once
    p.target[2, 1, 2400] = 0.5               # half is left to 1030
    p.target[2, 1, 1030] = 0.5
    p.uniform[2] = torch.tensor([0.9, 0.5, 0.0])
    p.target[3, 0] = p.draft[3, 0] = 0.5 * _certain(V, 7)   # u q < p holds
    p.target[4, 0] = 0.0                     # nothing at all: no token
    p.target[5, 0, 7] = 0.25                 # rejected by u = 0.25, and P - Q leaves nothing: P itself
    p.uniform[5] = torch.tensor([0.25, 0.0, 0.999])
    want = p.run()
    assert want[1].tolist() == [2499, 8, 1030, 2499, -1, 7]


def test_weights_that_are_not_numbers():
    """They count as 0, wherever they are."""
    _say("not finite")
    p = Problem(8, 4, 3000, "certain", seed=10)
    p.target[0, 0, 5:2000] = float("nan")
    p.target[1, :, 17] = float("inf")
    p.target[2, 0] = float("nan")
    p.target[3, :, ::2] = -1.0
    p.run()
    q = Problem(8, 4, 3000, "chain", seed=11)
    q.draft[0, 0] = float("nan")
    q.draft[1, :, 3:9] = float("inf")
    q.target[2, 0, 100:] = float("nan")
    q.run()


def test_a_token_tried_weighs_nothing():
    """Without a draft, next_token is never a child that was tried."""
    _say("removed")
    p = Problem(300, 4, 6, "tree", seed=12, sharp=3.0)
    p.parent[:] = torch.tensor([-1, 0, 0, 0], dtype=torch.int32)
    num, nxt, last, _ = p.run()
    for i in range(300):
        if last[i] == 0:
            assert int(nxt[i]) not in p.tokens[i, 1:].tolist()


def test_the_largest_vocabulary():
    _say("2^24")
    V = 2 ** 24
    p = Problem(1, 2, 8, "chain", seed=13)
    target, draft = torch.zeros(1, 2, V), torch.zeros(1, 1, V)
    target[0, :, V - 3:] = torch.tensor([0.25, 0.25, 0.5])
    draft[0, 0, 0] = 1.0
    p.vocab, p.target, p.draft = V, target, draft
    p.tokens = torch.tensor([[0, 0]], dtype=torch.int32)
    p.uniform = torch.tensor([[0.5, 0.6]])
    want = p.run()
    assert int(want[1][0]) == V - 1


def test_outputs_that_are_not_wanted_and_other_ways():
    _say("optional")
    p = Problem(9, 5, 2000, "chain", seed=14)
    want = p.expect()
    p.gpu()
    p.kw.update(window_index=None, path=None)
    p.call(stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(p.out[0].cpu(), want[0]) and torch.equal(p.out[1].cpu(), want[1])
    assert bool((p.out[2] == POISON).all()) and bool((p.path == POISON).all())
    p.out[0].fill_(POISON)
    p.call(workspace=torch.empty(1 << 16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(p.out[0].cpu(), want[0])


def test_no_slots_given():
    _say("no slots")
    p = Problem(9, 5, 200, "tree", seed=15)
    want = p.expect()
    p.gpu()
    p.kw["slot_idx"] = None
    p.call()
    p.check(want)


def test_captured_and_replayed():
    """Other tokens and numbers at each replay, eager calls between them."""
    _say("graph")
    ps = [Problem(16, 6, 3001, "chain", seed=20 + k, pads=(3,)) for k in range(3)]
    wants = [p.expect() for p in ps]
    p = ps[0]
    p.gpu()
    p.call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call()
    for k in (1, 2, 0):
        p.args[0].copy_(ps[k].tokens), p.args[1].copy_(ps[k].target), p.args[2].copy_(ps[k].uniform)
        p.kw["draft"].copy_(ps[k].draft)
        for t in p.out:
            t.fill_(POISON)
        p.path.fill_(POISON)
        graph.replay()
        p.check(wants[k])
        Problem(5, 4, 777, "tree", seed=k).run()
