"""The rest of a hybrid model's step, as cases that can be timed: layers whose state decays by
channel, rotated heads, and the verdict on the drafts.

Entry points of causal_conv1d_verify_amd that are covered:

* ``scan``    the selective state space scan over packed prompts (``selective_scan_prefill``):
              d = softplus(dt + dt_bias), h <- exp(d A) h + d B x, y = C h + D x, out = y silu(z);
* ``step``    the same recurrence for one new token per sequence (``selective_scan_update``);
* ``verify``  T draft tokens per sequence read against the state without changing it
              (``selective_scan_verify``), then the accepted ones folded into it
              (``selective_scan_commit``);
* ``rotary``  the RMS norm of each q and k head and the rotation by its token's position
              (``qk_norm_rotary``);
* ``accept``  drafts held against the target's probabilities with given random numbers, as a
              chain or as a tree, and the token behind the accepted ones (``accept_drafts``).

``run`` computes them with elementary torch operations in 32 bits (angles, probabilities and
their sums in 64) where ``own`` is false, and through the framework's entry points where it is
true.  ``exact`` computes them in 64 bits from the definitions, token by token.

Widths, heads, rows and draft lengths are those of the repository's workloads (8192, 10240 and
12288 channels, 16 q and k heads of 128, 8 x 17, 128 x 8 and 256 rows); 16 states a channel and
the vocabularies are generic.
"""

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # a small model in fp32: a few questions, one empty, one row a pad, an odd width and
        # more states than usual
        dict(name="scan_fp32_odd", op="scan", rows=5, longest=333, ragged=True, d=1048, n=24,
             x="f32", state="f32", pads=1, started=0.6, gate=True, skip=True, bias=True),
        # prompts of 2048 tokens, the width of the 8192-channel conv
        dict(name="scan_8x2048", op="scan", rows=8, longest=2048, ragged=False, d=8192, n=16,
             x="bf16", state="f32", pads=0, started=0.0, gate=True, skip=True, bias=True),
        # one long document alone on the card
        dict(name="scan_1x16384", op="scan", rows=1, longest=16384, ragged=False, d=4096, n=16,
             x="bf16", state="bf16", pads=0, started=0.0, gate=True, skip=True, bias=True),
        # one conversation that generates: latency
        dict(name="step_bs1", op="step", rows=1, T=1, d=8192, n=16, x="bf16", state="f32",
             pads=0, gate=True, skip=True, bias=True),
        # the 256-row batch of the 12288-channel conv, one token each
        dict(name="step_bs256", op="step", rows=256, T=1, d=12288, n=16, x="bf16", state="f32",
             pads=20, gate=True, skip=True, bias=True),
        # 17 draft tokens for each of 8 rows
        dict(name="verify_8x17", op="verify", rows=8, T=17, d=8192, n=16, x="bf16",
             state="bf16", pads=0, gate=True, skip=True, bias=True),
        # 8 draft tokens for each of 128 rows
        dict(name="verify_128x8", op="verify", rows=128, T=8, d=10240, n=16, x="bf16",
             state="f32", pads=9, gate=True, skip=True, bias=True),
        # q and k of one new token
        dict(name="rotary_bs1", op="rotary", tokens=1, hq=16, hk=16, dim=128, rot=128,
             x="bf16", norm=True, pairs=False, far=1000000),
        # q and k of 8 x 2048 prompt tokens, out of the rows of a wider projection; half of each
        # head is rotated
        dict(name="rotary_16384", op="rotary", tokens=16384, hq=16, hk=16, dim=128, rot=64,
             x="bf16", norm=True, pairs=False, far=100000),
        # the drafts of one conversation
        dict(name="accept_bs1", op="accept", rows=1, T=8, vocab=128000, p="f32", draft=True,
             tree=False, pads=0, short=False),
        # trees of 17 tokens for 8 rows, an odd vocabulary
        dict(name="accept_tree_8x17", op="accept", rows=8, T=17, vocab=50001, p="f32",
             draft=False, tree=True, pads=0, short=False),
        # 7 drafts for each of 128 rows, some rows with fewer
        dict(name="accept_128x8", op="accept", rows=128, T=8, vocab=128000, p="f32", draft=True,
             tree=False, pads=9, short=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _one(rng):
    op = rng.choice(["scan", "scan", "step", "verify", "rotary", "accept", "accept"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "step", "verify"):
        c = dict(op=op, rows=_log(rng, 1, 256 if op != "scan" else 24), d=8 * _log(rng, 4, 1536),
                 n=rng.choice([8, 16, 16, 16, 24, 32, 64]), x=x, state="f32" if x == "f32" else
                 rng.choice(["f32", "bf16"]), gate=rng.random() < 0.8, skip=rng.random() < 0.8,
                 bias=rng.random() < 0.8)
        c["pads"] = rng.randint(0, c["rows"] // 8)
        if op == "scan":
            c.update(longest=_log(rng, 1, 8192), ragged=rng.random() < 0.7,
                     started=rng.choice([0.0, 0.5, 1.0]))
        else:
            c["T"] = 1 if op == "step" else rng.randint(2, 32)
    elif op == "rotary":
        dim = 16 * rng.randint(2, 16)
        c = dict(op=op, tokens=_log(rng, 1, 16384), hq=rng.randint(1, 40), hk=rng.randint(1, 16),
                 dim=dim, rot=rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)]), x=x,
                 norm=rng.random() < 0.7, pairs=rng.random() < 0.3, far=_log(rng, 100, 4000000))
    else:
        tree = rng.random() < 0.4
        c = dict(op=op, rows=_log(rng, 1, 256), T=rng.randint(1, 32), vocab=_log(rng, 100, 160000),
                 p=rng.choice(["f32", "f32", "bf16"]), draft=not tree and rng.random() < 0.7,
                 tree=tree, short=rng.random() < 0.4)
        c["pads"] = rng.randint(0, c["rows"] // 8)
    return c


def draw(rng):
    # a fraction of the largest listed cases, so that a draw is never the costliest pass and
    # its probabilities are quickly made
    while True:
        c = _one(rng)
        w = work(c)
        states = c["rows"] * c.get("longest", c["T"] if c["op"] == "verify" else 1) * c["d"] * c["n"] \
            if "d" in c else 0
        probs = c["rows"] * c["T"] * c["vocab"] if c["op"] == "accept" else 0
        if w["bytes"] < 2e8 and states < 5e8 and probs < 1e8:
            return c


def _lengths(case):
    """Tokens of each prompt: the longest is there, an empty one too among ragged rows."""
    n, top = case["rows"], case["longest"]
    if not case["ragged"]:
        return [top] * n
    some = [(i * 7919 + 13 * n) % (top + 1) for i in range(n)]
    some[0] = top
    if n > 2:
        some[n // 2] = 0
    return some


def work(case):
    c = case
    if c["op"] in ("scan", "step", "verify"):
        x, s = BYTES[c["x"]], BYTES[c["state"]]
        live = c["rows"] - c["pads"]
        if c["op"] == "scan":
            # pads are the last rows
            tokens = sum(_lengths(c)[:live])
            states = live * (1 + c["started"])
        elif c["op"] == "step":
            tokens, states = live, 2 * live
        else:
            tokens, states = live * c["T"], 3 * live   # read; then read and written
        per = ((3 + c["gate"]) * c["d"] + 2 * c["n"]) * x
        area = c["d"] * c["n"]
        extra = 1.5 if c["op"] == "verify" else 1      # about half of the drafts again
        return {"bytes": tokens * per + states * area * s + 4 * area,
                "flops": 7.0 * tokens * area * extra}
    if c["op"] == "rotary":
        n = c["tokens"] * (c["hq"] + c["hk"]) * c["dim"]
        return {"bytes": 2 * n * BYTES[c["x"]] + 8 * c["tokens"], "flops": 9.0 * n}
    n = (c["rows"] - c["pads"]) * c["vocab"] * (1 + c["draft"])
    return {"bytes": n * BYTES[c["p"]] + 16 * c["rows"] * c["T"], "flops": 3.0 * n}


def prepare(case, seed):
    c = case
    gen = torch.Generator(DEVICE)
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEVICE)

    def slots(live):
        order = torch.randperm(live + 2, generator=gen, device=DEVICE)[:live]
        return torch.cat([order, order.new_full((c["pads"],), -1)]).to(torch.int32)

    if c["op"] == "rotary":
        # heads lie in rows q | k | v
        dt, n, dim = TYPES[c["x"]], c["tokens"], c["dim"]
        wide = (c["hq"] + c["hk"]) * dim
        rows = normal(n, wide + (wide // 2 + 7) // 8 * 8, dtype=dt)
        s = dict(c=c, rows=rows, q=rows[:, : c["hq"] * dim].unflatten(1, (c["hq"], dim)),
                 k=rows[:, c["hq"] * dim: wide].unflatten(1, (c["hk"], dim)),
                 wq=(1 + 0.1 * normal(dim)).to(dt) if c["norm"] else None,
                 wk=(1 + 0.1 * normal(dim)).to(dt) if c["norm"] else None)
        first = torch.randint(0, c["far"] + 1, (1,), generator=gen, device=DEVICE)
        s["qo"], s["ko"] = (torch.zeros(t.shape, dtype=dt, device=DEVICE) for t in (s["q"], s["k"]))
        s["positions"] = first + torch.arange(n, device=DEVICE)
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEVICE).float() / c["rot"])
        return s
    if c["op"] == "accept":
        n, T, V, dt = c["rows"], c["T"], c["vocab"], TYPES[c["p"]]
        logits = 3 * normal(n, T, V)
        s = dict(c=c, target=logits.softmax(-1).to(dt), draft=None, parent=None)
        if c["draft"]:
            guess = logits[:, : T - 1] + 0.8 * normal(n, T - 1, V)
            s["draft"] = guess.softmax(-1).to(dt)
            source = s["draft"]
        elif c["tree"]:
            back = (uniform(n, T) * 4).long() + 1
            parent = (torch.arange(T, device=DEVICE) - back).clamp(min=0)
            parent[:, 0] = -1
            s["parent"] = parent.to(torch.int32)
            source = s["target"].gather(1, parent[:, 1:, None].expand(-1, -1, V))
        else:
            source = s["target"][:, : T - 1]
        tokens = torch.randint(0, V, (n, T), generator=gen, device=DEVICE)
        if T > 1:
            tokens[:, 1:] = torch.multinomial(source.flatten(0, 1).float(), 1, generator=gen).view(n, T - 1)
        if c["short"]:                          # rows with fewer drafts end in -1
            there = 1 + (uniform(n, 1) * T).long()
            tokens = torch.where(torch.arange(T, device=DEVICE) < there, tokens, -1)
        s["tokens"] = tokens.to(torch.int32)
        s["uniform"] = uniform(n, T)
        s["slots"] = slots(n - c["pads"])
        s["num"], s["next"], s["last"] = (torch.zeros(n, dtype=torch.int32, device=DEVICE) for _ in range(3))
        s["path"] = torch.zeros(n, T, dtype=torch.int32, device=DEVICE)
        return s
    n, d, N, dt = c["rows"], c["d"], c["n"], TYPES[c["x"]]
    s = dict(c=c)
    if c["op"] == "scan":
        cu = [0]
        for t in _lengths(c):
            cu.append(cu[-1] + t)
        tokens = cu[-1]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEVICE)
        s["started"] = (uniform(n) < c["started"]).to(torch.int32)
    else:
        tokens = n * c["T"]
    # x as the conv leaves it; the gate beside it in the projection's rows; dt, B and C as the
    # projections behind the conv make them
    s["x"] = torch.nn.functional.silu(normal(tokens, d)).to(dt)
    s["z"] = normal(tokens, 2 * d, dtype=dt)[:, d:] if c["gate"] else None
    s["dt"] = (normal(tokens, d) - (0 if c["bias"] else 4.5)).to(dt)
    low = normal(tokens, 2 * N, dtype=dt)
    s["B"], s["C"] = low[:, :N], low[:, N:]
    s["out"] = torch.zeros(tokens, d, dtype=dt, device=DEVICE)
    # decays of 1 to N a unit of time, steps of 0.001 to 0.1 (and more) a token
    s["A"] = -(torch.arange(1, N + 1, device=DEVICE).float() * (0.9 + 0.2 * uniform(d, N)))
    s["D"] = 1 + 0.1 * normal(d) if c["skip"] else None
    s["dt_bias"] = normal(d) - 4.5 if c["bias"] else None
    live = n - c["pads"]
    s["slots"] = slots(live)
    s["live"] = torch.arange(live, device=DEVICE)
    s["pool"] = (0.1 * normal(live + 2, d, N)).to(TYPES[c["state"]])
    if c["op"] != "scan":
        for name in ("x", "z", "dt", "B", "C", "out"):
            s[name] = None if s[name] is None else s[name].unflatten(0, (n, c["T"]))
    if c["op"] == "verify":
        s["accepted"] = torch.randint(0, c["T"] + 1, (n,), generator=gen, device=DEVICE,
                                      dtype=torch.int32)
    return s


# ---- the plain forms -----------------------------------------------------------------


def _inclusive(a, b):
    """h of h_t = a_t h_{t-1} + b_t along dimension 1, from h = 0: pairs of tokens are made
    one, scanned, and taken apart again."""
    L = a.shape[1]
    if L == 1:
        return b
    even = L // 2 * 2
    a0, a1, b0, b1 = a[:, 0:even:2], a[:, 1:even:2], b[:, 0:even:2], b[:, 1:even:2]
    ends = _inclusive(a1 * a0, b1 + a1 * b0)
    h = torch.empty_like(b)
    h[:, 0] = b[:, 0]
    h[:, 1:even:2] = ends
    h[:, 2::2] = b[:, 2::2] + a[:, 2::2] * ends[:, : (L - 1) // 2]
    return h


def _delta(s, dt):
    v = dt.float() + (0 if s["dt_bias"] is None else s["dt_bias"])
    return v.clamp(min=0) + (-v.abs()).exp().log1p()


def _scanned(s, x, dt, z, B, C, first):
    """Outputs of [rows, L, d] tokens from the states `first` [rows, d, n], and the states
    behind every token."""
    x, B, C = x.float(), B.float(), C.float()
    delta = _delta(s, dt)
    a = (delta[..., None] * s["A"]).exp()
    b = (delta * x)[..., None] * B[:, :, None]
    b[:, 0] += a[:, 0] * first
    h = _inclusive(a, b)
    y = h.matmul(C[..., None])[..., 0]
    if s["D"] is not None:
        y = y + s["D"] * x
    if z is not None:
        y = y * (z.float() * z.float().sigmoid())
    return y, h


def _plain_scan(s):
    c, cu = s["c"], s["cu"].long()
    n, longest, tokens = c["rows"], c["longest"], s["x"].shape[0]
    at = torch.arange(longest, device=cu.device)
    there = at < (cu[1:] - cu[:-1])[:, None]
    idx = (cu[:-1, None] + at).clamp(max=tokens - 1)
    slots = s["slots"].long()
    first = s["pool"][slots.clamp(min=0)].float() * s["started"][:, None, None]
    y, h = _scanned(s, s["x"][idx], s["dt"][idx], None if s["z"] is None else s["z"][idx],
                    s["B"][idx], s["C"][idx], first)
    lengths = there.sum(1)
    last = h[torch.arange(n, device=cu.device), (lengths - 1).clamp(min=0)]
    last = torch.where((lengths > 0)[:, None, None], last, first)
    token = torch.arange(tokens, device=cu.device)
    row = torch.searchsorted(cu[1:], token, right=True)
    s["out"].copy_(torch.where((slots[row] >= 0)[:, None], y[row, token - cu[row]].to(s["out"].dtype), s["out"]))
    live = s["live"]
    s["pool"][slots[live]] = last[live].to(s["pool"].dtype)
    return s["out"], s["pool"]


def _plain_few(s):
    live = s["live"]
    slots = s["slots"][live].long()
    first = s["pool"][slots].float()
    y, h = _scanned(s, s["x"][live], s["dt"][live], None if s["z"] is None else s["z"][live],
                    s["B"][live], s["C"][live], first)
    s["out"][live] = y.to(s["out"].dtype)
    if s["c"]["op"] == "verify":
        taken = s["accepted"][live].long()
        after = torch.where((taken > 0)[:, None, None], h[live, (taken - 1).clamp(min=0)], first)
    else:
        after = h[:, -1]
    s["pool"][slots] = after.to(s["pool"].dtype)
    return s["out"], s["pool"]


def _rotated(x, w, angle, pairs):
    y = x.float()
    if w is not None:
        y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float()
    r = angle.shape[-1]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = (y[..., 0:2 * r:2], y[..., 1:2 * r:2]) if pairs else (y[..., :r], y[..., r:2 * r])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., 2 * r:]], -1).to(x.dtype)


def _plain_rotary(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    pairs = s["c"]["pairs"]
    return _rotated(s["q"], s["wq"], angle, pairs), _rotated(s["k"], s["wk"], angle, pairs)


def _reached(edges):
    """Which nodes lie on the way from node 0 along `edges` [rows, T, T] (parent, child)."""
    T = edges.shape[1]
    hops = edges.double() + torch.eye(T, device=edges.device, dtype=torch.float64)
    for _ in range(max(1, (T - 1).bit_length())):
        hops = hops.matmul(hops.contiguous()).clamp(max=1)
    return hops[:, 0] > 0


def _plain_accept(s):
    c, T, V = s["c"], s["c"]["T"], s["c"]["vocab"]
    n = c["rows"]
    dev = s["tokens"].device
    x = s["tokens"][:, 1:].long()
    node = torch.arange(T, device=dev)
    parent = s["parent"][:, 1:].long() if c["tree"] else node[:-1].expand(n, -1)
    valid = x >= 0
    at = x.clamp(min=0)
    rows = torch.arange(n, device=dev)
    p = torch.where(valid, s["target"][rows[:, None], parent, at].double(), 0)
    # the mass that is left behind the siblings before each node
    before = (parent[:, :, None] == parent[:, None, :]) & (node[1:, None] > node[None, 1:])
    same = before & (x[:, :, None] == x[:, None, :])
    first = valid & ~same.any(-1)
    gone = (before.double() * (p * first)[:, None, :]).sum(-1)
    q = s["draft"][rows[:, None], parent, at].double() if c["draft"] else 1 - gone
    ok = first & (s["uniform"][:, :-1].double() * q < p)
    chosen = ok & ~(before & ok[:, None, :]).any(-1)
    edges = torch.zeros(n, T, T, dtype=torch.bool, device=dev)
    edges[:, :, 1:] = chosen[:, None] & (parent[:, None] == node[:, None])
    reached = _reached(edges)
    num = reached.sum(1)
    last = (reached * node).amax(1)
    path = torch.where(reached, node, T).sort(1)[0]
    path = torch.where(path < T, path, -1)
    # what the next token is drawn from
    w = s["target"][rows, last].double()
    child = (parent == last[:, None]) & valid
    if c["draft"]:
        d = s["draft"][rows, last.clamp(max=max(T - 2, 0))].double() if T > 1 else 0
        rest = (w - d).clamp(min=0)
        rest = torch.where(child.any(1, keepdim=True), rest, w)
    else:
        rest = torch.cat([w, w.new_zeros(n, 1)], 1).scatter(1, torch.where(child, at, V), 0)[:, :V]
    rest = torch.where((rest > 0).any(1, keepdim=True), rest, w)
    upto = rest.cumsum(1)
    over = upto > s["uniform"][:, -1:].double() * upto[:, -1:]
    final = V - 1 - (rest > 0).flip(1).int().argmax(1)
    token = torch.where(over.any(1), over.int().argmax(1), final)
    live = s["slots"] >= 0
    for name, v in (("num", num), ("next", token), ("last", last), ("path", path)):
        s[name].copy_(torch.where(live if v.dim() == 1 else live[:, None], v.to(torch.int32), s[name]))
    return s["num"], s["next"], s["last"], s["path"]


# ---- the framework's calls -----------------------------------------------------------


def _own(s):
    import causal_conv1d_verify_amd as cv

    op = s["c"]["op"]
    if op == "scan":
        cv.selective_scan_prefill(s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"], s["out"],
                                  s["cu"], max_len=s["c"]["longest"], z=s["z"], D=s["D"],
                                  dt_bias=s["dt_bias"], slot_idx=s["slots"],
                                  has_initial_state=s["started"])
        return s["out"], s["pool"]
    if op == "step":
        cv.selective_scan_update(s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"], s["out"],
                                 z=s["z"], D=s["D"], dt_bias=s["dt_bias"], slot_idx=s["slots"])
        return s["out"], s["pool"]
    if op == "verify":
        cv.selective_scan_verify(s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"], s["out"],
                                 z=s["z"], D=s["D"], dt_bias=s["dt_bias"], slot_idx=s["slots"])
        cv.selective_scan_commit(s["x"], s["dt"], s["A"], s["B"], s["pool"], s["accepted"],
                                 dt_bias=s["dt_bias"], slot_idx=s["slots"])
        return s["out"], s["pool"]
    if op == "rotary":
        cv.qk_norm_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], s["qo"], s["ko"],
                          q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=s["c"]["pairs"])
        return s["qo"], s["ko"]
    cv.accept_drafts(s["tokens"], s["target"], s["uniform"], s["num"], s["next"],
                     draft=s["draft"], parent=s["parent"], window_index=s["last"], path=s["path"],
                     slot_idx=s["slots"])
    return s["num"], s["next"], s["last"], s["path"]


def run(state):
    if own:
        return _own(state)
    plain = {"scan": _plain_scan, "step": _plain_few, "verify": _plain_few,
             "rotary": _plain_rotary, "accept": _plain_accept}[state["c"]["op"]]
    return plain(state)


# ---- 64 bits, from the definitions ---------------------------------------------------


def _exact_accept(s):
    c, T, V = s["c"], s["c"]["T"], s["c"]["vocab"]
    num, nxt, last, path = (s[k].cpu().clone() for k in ("num", "next", "last", "path"))
    tokens, u, slots = s["tokens"].cpu(), s["uniform"].double().cpu(), s["slots"].cpu()
    parent = s["parent"].cpu() if c["tree"] else None
    for i in range(c["rows"]):
        if slots[i] < 0:
            continue
        at, way = 0, [0]
        left, gone, drafted = 1.0, [], False
        p = s["target"][i, 0].double().cpu()
        for j in range(1, T):
            if (int(parent[i, j]) if c["tree"] else j - 1) != at:
                continue
            x = int(tokens[i, j])
            if x < 0:
                continue
            if x not in gone:
                q = float(s["draft"][i, at, x]) if c["draft"] else left
                if float(u[i, j - 1]) * q < float(p[x]):
                    at, left, gone, drafted = j, 1.0, [], False
                    way.append(j)
                    p = s["target"][i, j].double().cpu()
                    continue
                left -= float(p[x])
                gone.append(x)
            drafted = True
        w = p.clone()
        if drafted and c["draft"]:
            w = (p - s["draft"][i, at].double().cpu()).clamp(min=0)
        elif drafted:
            w[gone] = 0
        if not bool((w > 0).any()):
            w = p
        sums = w.cumsum(0)
        over = (sums > u[i, T - 1] * sums[-1]).nonzero()
        num[i], last[i] = len(way), at
        nxt[i] = int(over[0]) if len(over) else int((w > 0).nonzero()[-1])
        path[i] = torch.tensor(way + [-1] * (T - len(way)), dtype=torch.int32)
    return num, nxt, last, path


def exact(case, seed):
    s = prepare(case, seed)
    c, op, f64 = case, case["op"], torch.float64
    if op == "accept":
        return _exact_accept(s)
    if op == "rotary":
        outs = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            y = x.to(f64)
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["dim"] + EPS) * w.to(f64)
            o = y.clone()
            for i in range(c["rot"] // 2):
                e, f = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + c["rot"] // 2)
                a = (s["positions"].to(f64) * s["inv_freq"][i].to(f64))[:, None]
                o[..., e] = y[..., e] * torch.cos(a) - y[..., f] * torch.sin(a)
                o[..., f] = y[..., f] * torch.cos(a) + y[..., e] * torch.sin(a)
            outs.append(o)
        return tuple(outs)
    live = c["rows"] - c["pads"]
    pool, out = s["pool"].to(f64), s["out"].to(f64)
    slots = s["slots"][:live].long()
    A, zero = s["A"].to(f64), torch.zeros((), dtype=f64, device=DEVICE)
    bias = zero if s["dt_bias"] is None else s["dt_bias"].to(f64)
    skip = zero if s["D"] is None else s["D"].to(f64)

    def token(h, x, dt, z, B, C):
        x, v = x.to(f64), dt.to(f64) + bias
        d = torch.where(v > 30, v, torch.log1p(torch.exp(v.clamp(max=30))))
        h = h * torch.exp(d[..., None] * A) + (d * x)[..., None] * B.to(f64)[..., None, :]
        y = (h * C.to(f64)[..., None, :]).sum(-1) + skip * x
        if z is not None:
            y = y * z.to(f64) / (1 + torch.exp(-z.to(f64)))
        return h, y

    h = pool[slots]
    gate = (lambda at: None) if s["z"] is None else (lambda at: s["z"][at])
    if op == "scan":
        h = h * s["started"][:live, None, None]
        lengths = _lengths(c)[:live]
        start = s["cu"][:live].long()
        # rows by falling length, so that the rows that still hold a token are the first ones
        order = sorted(range(live), key=lambda i: -lengths[i])
        by = torch.tensor(order, device=DEVICE)
        h, start = h[by], start[by]
        m = live
        for t in range(max(lengths, default=0)):
            while m and lengths[order[m - 1]] <= t:
                m -= 1
            at = start[:m] + t
            h[:m], out[at] = token(h[:m], s["x"][at], s["dt"][at], gate(at), s["B"][at], s["C"][at])
        back = torch.empty_like(h)
        back[by] = h
        pool[slots] = back
        return out, pool
    after = h.clone()
    for t in range(c["T"]):
        at = (slice(0, live), t)
        h, out[at] = token(h, s["x"][at], s["dt"][at], gate(at), s["B"][at], s["C"][at])
        if op == "verify":
            after = torch.where((s["accepted"][:live] > t)[:, None, None], h, after)
    pool[slots] = after if op == "verify" else h
    return out, pool
