"""The operators that follow the conv of a linear-attention layer, as cases that can be timed.

Six entry points of causal_conv1d_verify_amd are covered, in the order in which a layer
calls them behind its conv:

* ``prefill``  linear attention with a decay for each head over packed prompts
               (``linear_attn_prefill``): S <- exp(g) S + k v^T, o = scale * S^T q;
* ``decode``   the same recurrence for one new token per sequence (``linear_attn_update``);
* ``verify``   T draft tokens per sequence read against the state without changing it
               (``linear_attn_verify``), then the accepted ones folded into it
               (``linear_attn_commit``);
* ``gate``     the per-head RMS norm of the attention's output with its gate
               (``gated_norm``);
* ``residual`` the norm after a block, its gate, the scaled residual sum and the norm before
               the next block (``residual_norm``).

``run`` computes them with elementary torch operations in 32 bits (decays are summed in 64)
where ``own`` is false, and through the framework's entry points where it is true.
``exact`` computes them in 64 bits from the definitions, token by token.

Head counts and sizes are those of the repository's workloads: 16 q and k heads with 48 or
32 v heads (10240 and 8192 conv channels), 32 of each (12288), all of 128 channels; rows,
draft lengths and state types are theirs too.
"""

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
CHUNK = 64
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a few short questions that arrive together, one of them empty and one row a pad
        dict(name="prefill_short", op="prefill", rows=8, longest=160, ragged=True, hq=16, hv=48,
             dk=128, dv=128, x="bf16", state="f32", decay="token", pads=1, started=0.5),
        # prompts of 2048 tokens, the width of the 10240-channel conv
        dict(name="prefill_8x2048", op="prefill", rows=8, longest=2048, ragged=False, hq=16,
             hv=48, dk=128, dv=128, x="bf16", state="f32", decay="token", pads=0, started=0.0),
        # one long document alone on the card, the width of the 8192-channel conv
        dict(name="prefill_1x16384", op="prefill", rows=1, longest=16384, ragged=False, hq=16,
             hv=32, dk=128, dv=128, x="bf16", state="bf16", decay="token", pads=0, started=0.0),
        # a small model in fp32 with heads off the powers of two and constant decays
        dict(name="prefill_fp32_odd", op="prefill", rows=5, longest=777, ragged=True, hq=2,
             hv=6, dk=96, dv=72, x="f32", state="f32", decay="head", pads=0, started=0.6),
        # one conversation that generates: latency
        dict(name="decode_bs1", op="decode", rows=1, T=1, hq=16, hv=48, dk=128, dv=128,
             x="bf16", state="f32", decay="token", pads=0),
        # the 256-row batch of the 12288-channel conv, one token each
        dict(name="decode_bs256", op="decode", rows=256, T=1, hq=32, hv=32, dk=128, dv=128,
             x="bf16", state="f32", decay="token", pads=20),
        # 17 draft tokens for each of 8 rows
        dict(name="verify_8x17", op="verify", rows=8, T=17, hq=16, hv=32, dk=128, dv=128,
             x="bf16", state="bf16", decay="token", pads=0),
        # 8 draft tokens for each of 128 rows
        dict(name="verify_128x8", op="verify", rows=128, T=8, hq=16, hv=48, dk=128, dv=128,
             x="bf16", state="f32", decay="token", pads=9),
        # the gated head norm behind a single-token step, and behind the 8 x 2048 prompts
        dict(name="gate_bs1", op="gate", rows=1, heads=48, dim=128, x="bf16", act="silu",
             first=False),
        dict(name="gate_16384", op="gate", rows=16384, heads=48, dim=128, x="bf16",
             act="silu", first=False),
        # the block's end: a verify step of 128 x 8 tokens, and long prompts with an fp32
        # residual stream and a gate for each token
        dict(name="residual_1024", op="residual", rows=1024, dim=5120, x="bf16", res="bf16",
             post=True, gate="none", scale=1.0),
        dict(name="residual_16384", op="residual", rows=16384, dim=4096, x="bf16", res="f32",
             post=True, gate="token", scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _one(rng):
    op = rng.choice(["prefill", "prefill", "decode", "verify", "gate", "residual"])
    if op in ("prefill", "decode", "verify"):
        x = rng.choice(["bf16", "bf16", "bf16", "f32"])
        hq = rng.choice([1, 2, 3, 4, 8, 16, 32])
        c = dict(op=op, rows=_log(rng, 1, 256 if op != "prefill" else 24), hq=hq,
                 hv=min(64, hq * rng.choice([1, 1, 2, 3, 4])), dk=8 * rng.randint(4, 24),
                 dv=8 * rng.randint(4, 24), x=x, state="f32" if x == "f32" else
                 rng.choice(["f32", "bf16"]), decay=rng.choice(["token", "token", "head"]))
        if rng.random() < 0.5:
            c["dk"] = c["dv"] = rng.choice([64, 128, 128, 256])
        c["hv"] -= c["hv"] % hq
        c["pads"] = rng.randint(0, c["rows"] // 8)
        if op == "prefill":
            c.update(longest=_log(rng, 1, 8192), ragged=rng.random() < 0.7,
                     started=rng.choice([0.0, 0.5, 1.0]))
        else:
            c["T"] = 1 if op == "decode" else rng.randint(2, 32)
    elif op == "gate":
        c = dict(op=op, rows=_log(rng, 1, 16384), heads=rng.randint(1, 64),
                 dim=8 * rng.randint(4, 40), x=rng.choice(["bf16", "f32"]),
                 act=rng.choice(["silu", "sigmoid"]), first=rng.random() < 0.4)
    else:
        x = rng.choice(["bf16", "bf16", "f32"])
        c = dict(op=op, rows=_log(rng, 1, 16384), dim=8 * _log(rng, 8, 1024), x=x,
                 res="f32" if x == "f32" else rng.choice(["bf16", "f32"]),
                 post=rng.random() < 0.6, gate=rng.choice(["none", "token", "channel"]),
                 scale=rng.choice([1.0, 0.5, 0.22]))
    return c


def draw(rng):
    # nothing over half of the largest listed prompt batch, so that a draw is never the
    # costliest pass (ragged rows pad to the longest one in the plain form)
    while True:
        c = _one(rng)
        w = work(c)
        padded = c["rows"] * c.get("longest", 0) * c.get("hv", 0) * max(c.get("dk", 0), c.get("dv", 0))
        if w["bytes"] < 4e8 and w["flops"] < 2.5e10 and padded < 6e7:
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
    c, b = case, {"bf16": 2, "f32": 4}
    if c["op"] in ("prefill", "decode", "verify"):
        x, s = b[c["x"]], b[c["state"]]
        live = c["rows"] - c["pads"]
        if c["op"] == "prefill":
            # pads are the last rows
            tokens = sum(_lengths(c)[:live])
            states = live * (1 + c["started"])
        elif c["op"] == "decode":
            tokens, states = live, 2 * live
        else:
            tokens, states = live * c["T"], 3 * live   # read; then read and written
        per = (2 * c["hq"] * c["dk"] + 2 * c["hv"] * c["dv"]) * x
        per += 4 * c["hv"] if c["decay"] == "token" else 0
        area = c["hv"] * c["dk"] * c["dv"]
        extra = 1.5 if c["op"] == "verify" else 1      # about half of the drafts again
        return {"bytes": tokens * per + states * area * s, "flops": 4.0 * tokens * area * extra}
    if c["op"] == "gate":
        n = c["rows"] * c["heads"] * c["dim"]
        return {"bytes": 3 * n * b[c["x"]] + c["dim"] * b[c["x"]], "flops": 12.0 * n}
    n = c["rows"] * c["dim"]
    gate = {"none": 0, "token": n, "channel": c["dim"]}[c["gate"]]
    return {"bytes": (2 * n + gate + 2 * c["dim"]) * b[c["x"]] + 2 * n * b[c["res"]],
            "flops": 10.0 * n}


def prepare(case, seed):
    c = case
    gen = torch.Generator(DEVICE)
    gen.manual_seed(int(seed))
    dt = TYPES[c["x"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)

    if c["op"] == "gate":
        shape = (c["rows"], c["heads"], c["dim"])
        return dict(c=c, y=normal(*shape, dtype=dt), z=normal(*shape, dtype=dt),
                    w=(1 + 0.1 * normal(c["dim"])).to(dt), out=torch.zeros(shape, dtype=dt, device=DEVICE))
    if c["op"] == "residual":
        shape = (c["rows"], c["dim"])
        gate = {"none": lambda: None, "token": lambda: normal(*shape, dtype=dt),
                "channel": lambda: normal(c["dim"], dtype=dt)}[c["gate"]]()
        return dict(c=c, y=normal(*shape, dtype=dt), res=3 * normal(*shape, dtype=TYPES[c["res"]]),
                    gate=gate, w_post=(1 + 0.1 * normal(c["dim"])).to(dt) if c["post"] else None,
                    w_pre=(1 + 0.1 * normal(c["dim"])).to(dt),
                    res_out=torch.zeros(shape, dtype=TYPES[c["res"]], device=DEVICE),
                    out=torch.zeros(shape, dtype=dt, device=DEVICE))
    hq, hv, dk, dv, n = c["hq"], c["hv"], c["dk"], c["dv"], c["rows"]
    s = dict(c=c)
    if c["op"] == "prefill":
        lengths = _lengths(c)
        cu = [0]
        for t in lengths:
            cu.append(cu[-1] + t)
        tokens = cu[-1]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEVICE)
        s["started"] = (torch.rand(n, generator=gen, device=DEVICE) < c["started"]).to(torch.int32)
    else:
        tokens = n * c["T"]
    # one row of q | k | v channels for each token, as the conv leaves it: SiLU of the conv,
    # q and k normalised by head
    qkv = torch.nn.functional.silu(normal(tokens, 2 * hq * dk + hv * dv))
    heads = qkv[:, : 2 * hq * dk].view(tokens, 2 * hq, dk)
    heads /= heads.square().sum(-1, keepdim=True).add(EPS).sqrt()
    qkv = qkv.to(dt)
    s["q"] = qkv[:, : hq * dk].unflatten(1, (hq, dk))
    s["k"] = qkv[:, hq * dk: 2 * hq * dk].unflatten(1, (hq, dk))
    s["v"] = qkv[:, 2 * hq * dk:].unflatten(1, (hv, dv))
    # decays: a rate of 1 to 16 for each head times a step of 0.001 to 0.1 (or more) a token
    rate = 1 + 15 * torch.rand(hv, generator=gen, device=DEVICE)
    step = torch.nn.functional.softplus(normal(tokens if c["decay"] == "token" else 1, hv) - 4.0)
    s["g"] = -(rate * step) if c["decay"] == "token" else -(rate * step)[0]
    s["out"] = torch.zeros(tokens, hv, dv, dtype=dt, device=DEVICE)
    # the pool has two slots more than live rows; pads are the last rows
    live = n - c["pads"]
    order = torch.randperm(live + 2, generator=gen, device=DEVICE)[:live]
    s["slots"] = torch.cat([order, order.new_full((c["pads"],), -1)]).to(torch.int32)
    s["live"] = torch.arange(live, device=DEVICE)
    s["pool"] = (0.1 * normal(live + 2, hv, dk, dv)).to(TYPES[c["state"]])
    if c["op"] != "prefill":
        for name in ("q", "k", "v", "out"):
            s[name] = s[name].unflatten(0, (n, c["T"]))
        if c["decay"] == "token":
            s["g"] = s["g"].unflatten(0, (n, c["T"]))
        if c["op"] == "verify":
            s["accepted"] = torch.randint(0, c["T"] + 1, (n,), generator=gen, device=DEVICE,
                                          dtype=torch.int32)
    return s


# ---- the plain forms -----------------------------------------------------------------


def _chunked(q, k, v, g, first, scale):
    """Decayed linear attention over [B, L, H, D] rows of whole chunks, from the states
    `first` [B, H, dk, dv]: the outputs and the states after the last token."""
    B, L, H, dv = v.shape
    n = L // CHUNK

    def chunks(x):
        return x.unflatten(1, (n, CHUNK)).permute(0, 3, 1, 2, *range(4, x.dim() + 1))

    q, k, v, g = (chunks(x) for x in (q, k, v, g))           # [B, H, n, CHUNK, ...]
    G = g.double().cumsum(-1)
    below = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    decay = (G[..., :, None] - G[..., None, :]).masked_fill(~below, -math.inf).exp().float()
    o = (torch.matmul(q, k.transpose(-1, -2)) * decay).matmul(v)
    left = (G[..., -1:] - G).exp().float()[..., None]
    added = torch.matmul((k * left).transpose(-1, -2), v)    # what each chunk adds
    # the state that enters chunk c: the first one and what chunks before c added, decayed
    T = torch.nn.functional.pad(G[..., -1].cumsum(-1), (1, 0))
    before = torch.ones(n + 1, n + 1, dtype=torch.bool, device=v.device).tril()
    M = (T[..., :, None] - T[..., None, :]).masked_fill(~before, -math.inf).exp().float()
    enters = M.matmul(torch.cat([first[:, :, None], added], 2).flatten(3)).unflatten(3, first.shape[2:])
    o = o + torch.matmul(q * G.exp().float()[..., None], enters[:, :, :n])
    return (scale * o).permute(0, 2, 3, 1, 4).reshape(B, L, H, dv), enters[:, :, n]


def _plain_prefill(s):
    c, cu = s["c"], s["cu"].long()
    n, tokens, rep = c["rows"], s["v"].shape[0], c["hv"] // c["hq"]
    longest = -(-c["longest"] // CHUNK) * CHUNK
    at = torch.arange(longest, device=cu.device)
    there = at < (cu[1:] - cu[:-1])[:, None]
    idx = (cu[:-1, None] + at).clamp(max=tokens - 1)

    def rows(x, heads):
        x = torch.where(there.reshape(n, longest, *[1] * (x.dim() - 1)), x[idx], 0)
        return (x if x.dtype == torch.float64 else x.float()).repeat_interleave(heads, 2)

    g = s["g"].double().expand(tokens, c["hv"])
    slots = s["slots"].long()
    first = s["pool"][slots.clamp(min=0)].float() * s["started"][:, None, None, None]
    o, last = _chunked(rows(s["q"], rep), rows(s["k"], rep), rows(s["v"], 1), rows(g, 1), first,
                       c["dk"] ** -0.5)
    token = torch.arange(tokens, device=cu.device)
    row = torch.searchsorted(cu[1:], token, right=True)
    s["out"].copy_(torch.where((slots[row] >= 0)[:, None, None], o[row, token - cu[row]].to(s["out"].dtype), s["out"]))
    live = s["live"]
    s["pool"][slots[live]] = last[live].to(s["pool"].dtype)
    return s["out"], s["pool"]


def _few(s):
    """Rows of T tokens as 32-bit [B, H, T, D] of the live rows, and their log decays."""
    live, rep = s["live"], s["c"]["hv"] // s["c"]["hq"]
    q, k = (x[live].float().repeat_interleave(rep, 2).transpose(1, 2) for x in (s["q"], s["k"]))
    v = s["v"][live].float().transpose(1, 2)
    g = s["g"].double().expand(s["v"].shape[:3])[live].transpose(1, 2)
    return q, k, v, g, s["slots"][live].long()


def _plain_decode(s):
    q, k, v, g, slots = _few(s)
    S = s["pool"][slots].float() * g.exp().float()[..., None] + k.transpose(-1, -2) * v
    s["out"][s["live"]] = (s["c"]["dk"] ** -0.5 * q.matmul(S)).transpose(1, 2).to(s["out"].dtype)
    s["pool"][slots] = S.to(s["pool"].dtype)
    return s["out"], s["pool"]


def _plain_verify(s):
    q, k, v, g, slots = _few(s)
    T = s["c"]["T"]
    S = s["pool"][slots].float()
    G = g.cumsum(-1)
    below = torch.ones(T, T, dtype=torch.bool, device=v.device).tril()
    decay = (G[..., :, None] - G[..., None, :]).masked_fill(~below, -math.inf).exp().float()
    o = (q.matmul(k.transpose(-1, -2)) * decay).matmul(v) + (q * G.exp().float()[..., None]).matmul(S)
    s["out"][s["live"]] = (s["c"]["dk"] ** -0.5 * o).transpose(1, 2).to(s["out"].dtype)
    # the accepted tokens
    taken = s["accepted"][s["live"]].long()[:, None, None]
    G = torch.nn.functional.pad(G, (1, 0))
    total = G.gather(-1, taken.expand(-1, G.shape[1], 1))
    left = torch.where(torch.arange(T, device=v.device) < taken, (total - G[..., 1:]).clamp(max=0).exp(), 0).float()
    S = S * total.exp().float()[..., None] + (k * left[..., None]).transpose(-1, -2).matmul(v)
    s["pool"][slots] = S.to(s["pool"].dtype)
    return s["out"], s["pool"]


def _act(z, act):
    return z * z.sigmoid() if act == "silu" else z.sigmoid()


def _rms(x, w):
    return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.to(x.dtype)


def _plain_gate(s):
    c, y, a = s["c"], s["y"].float(), _act(s["z"].float(), s["c"]["act"])
    o = _rms(y * a, s["w"]) if c["first"] else _rms(y, s["w"]) * a
    return o.to(s["y"].dtype)


def _plain_residual(s):
    u = s["y"].float()
    if s["w_post"] is not None:
        u = _rms(u, s["w_post"])
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["res"].float() + s["c"]["scale"] * u
    return r.to(s["res"].dtype), _rms(r, s["w_pre"]).to(s["y"].dtype)


# ---- the framework's calls -----------------------------------------------------------


def _own(s):
    import causal_conv1d_verify_amd as cv

    op = s["c"]["op"]
    if op == "prefill":
        cv.linear_attn_prefill(s["q"], s["k"], s["v"], s["g"], s["pool"], s["out"], s["cu"],
                               max_len=s["c"]["longest"], slot_idx=s["slots"],
                               has_initial_state=s["started"])
        return s["out"], s["pool"]
    if op == "decode":
        cv.linear_attn_update(s["q"], s["k"], s["v"], s["g"], s["pool"], s["out"],
                              slot_idx=s["slots"])
        return s["out"], s["pool"]
    if op == "verify":
        cv.linear_attn_verify(s["q"], s["k"], s["v"], s["g"], s["pool"], s["out"],
                              slot_idx=s["slots"])
        cv.linear_attn_commit(s["k"], s["v"], s["g"], s["pool"], s["accepted"],
                              slot_idx=s["slots"])
        return s["out"], s["pool"]
    if op == "gate":
        cv.gated_norm(s["y"], s["z"], s["w"], s["out"], eps=EPS, activation=s["c"]["act"],
                      gate_first=s["c"]["first"])
        return s["out"]
    cv.residual_norm(s["y"], s["res"], s["w_pre"], s["out"], post_weight=s["w_post"],
                     gate=s["gate"], scale=s["c"]["scale"], residual_out=s["res_out"], eps=EPS)
    return s["res_out"], s["out"]


def run(state):
    if own:
        return _own(state)
    plain = {"prefill": _plain_prefill, "decode": _plain_decode, "verify": _plain_verify,
             "gate": _plain_gate, "residual": _plain_residual}[state["c"]["op"]]
    return plain(state)


# ---- 64 bits, from the definitions ---------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    f64 = torch.float64
    if op == "gate":
        y, z = s["y"].to(f64), s["z"].to(f64)
        a = 1 / (1 + torch.exp(-z))
        if c["act"] == "silu":
            a = a * z
        if c["first"]:
            y = y * a
        o = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["dim"] + EPS) * s["w"].to(f64)
        return o if c["first"] else o * a
    if op == "residual":
        u = s["y"].to(f64)
        if c["post"]:
            u = u / torch.sqrt((u * u).sum(-1, keepdim=True) / c["dim"] + EPS) * s["w_post"].to(f64)
        if s["gate"] is not None:
            u = u * s["gate"].to(f64)
        r = s["res"].to(f64) + c["scale"] * u
        return r, r / torch.sqrt((r * r).sum(-1, keepdim=True) / c["dim"] + EPS) * s["w_pre"].to(f64)
    live, hv, dk, dv = c["rows"] - c["pads"], c["hv"], c["dk"], c["dv"]
    group = torch.arange(hv, device=DEVICE) // (hv // c["hq"])
    pool, out = s["pool"].to(f64), s["out"].to(f64)
    g = s["g"].to(f64)
    slots = s["slots"][:live].long()
    S = pool[slots]
    if op == "prefill":
        S = S * s["started"][:live, None, None, None]
        lengths = _lengths(c)[:live]
        start = s["cu"][:live].long()
        # rows by falling length, so that the rows that still hold a token are the first ones
        order = sorted(range(live), key=lambda i: -lengths[i])
        by = torch.tensor(order, device=DEVICE)
        S, start = S[by], start[by]
        m = live
        for t in range(max(lengths, default=0)):
            while m and lengths[order[m - 1]] <= t:
                m -= 1
            at = start[:m] + t
            a = torch.exp(g[at] if c["decay"] == "token" else g.expand(m, hv))
            kt, vt, qt = s["k"][at].to(f64)[:, group], s["v"][at].to(f64), s["q"][at].to(f64)[:, group]
            S[:m] = S[:m].mul_(a[..., None, None]).add_(kt[..., :, None] * vt[..., None, :])
            out[at] = (qt[..., None, :] @ S[:m])[..., 0, :] / math.sqrt(dk)
        back = torch.empty_like(S)
        back[by] = S
        pool[slots] = back
        return out, pool
    after = S.clone()
    for t in range(c["T"]):
        a = torch.exp(g[:live, t] if c["decay"] == "token" else g.expand(live, hv))[..., None, None]
        kt, vt, qt = s["k"][:live, t].to(f64)[:, group], s["v"][:live, t].to(f64), s["q"][:live, t].to(f64)[:, group]
        S = S * a + kt[..., :, None] * vt[..., None, :]
        out[:live, t] = (qt[..., None, :] @ S)[..., 0, :] / math.sqrt(dk)
        if op == "verify":
            more = (s["accepted"][:live] > t)[:, None, None, None]
            after = torch.where(more, S, after)
    pool[slots] = after if op == "verify" else S
    return out, pool
