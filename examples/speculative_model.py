"""A small hybrid model that writes with drafts, on the framework's kernels: a selective scan behind its
conv, then linear attention over rotated heads, then a head over a vocabulary.

    prompt   conv_prefill -> selective_scan_prefill; qk_norm_rotary -> linear_attn_prefill
    verify   conv_verify_update_dedup -> selective_scan_verify; qk_norm_rotary -> linear_attn_verify
    verdict  accept_drafts: what is kept of the drafts, and the token behind them
    commit   conv_verify_restore, selective_scan_commit, linear_attn_commit, all from the verdict's own
             tensors: the host is not asked

The projections are torch products, the drafts come from a table of which token follows which.  Run as
a program it writes a few steps, and compares the model's probabilities for what comes next with those
of one long prompt over everything that was kept:

    python examples/speculative_model.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_conv1d_verify_amd as cv  # noqa: E402

BF16 = torch.bfloat16


class SpeculativeModel:
    def __init__(self, vocab=500, dim=256, d_inner=512, d_state=16, heads=4, head_dim=64, rot=32, T=6, slots=8, d_conv=4,
                 device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)

        def weight(*shape, scale=None):
            return ((shape[0] ** -0.5 if scale is None else scale) *
                    torch.randn(*shape, generator=gen, device=device)).to(BF16)

        self.vocab, self.T, self.d_state, self.heads, self.head_dim, self.d_conv = vocab, T, d_state, heads, head_dim, d_conv
        self.embed = weight(vocab, dim, scale=0.3)
        # the scan's layer
        self.w_x, self.w_z = weight(dim, d_inner), weight(dim, d_inner)
        self.w_conv = weight(d_inner, d_conv, scale=0.5)
        self.w_low, self.w_dt = weight(d_inner, 16 + 2 * d_state), weight(16, d_inner)
        self.dt_bias = torch.randn(d_inner, generator=gen, device=device) - 4
        self.A = -torch.arange(1, d_state + 1, device=device).float().repeat(d_inner, 1)
        self.D = torch.ones(d_inner, device=device)
        self.w_scan = weight(d_inner, dim, scale=3.0 * d_inner ** -0.5)
        self.conv_state = torch.zeros(slots, d_inner, d_conv - 1, dtype=BF16, device=device)
        self.windows = torch.zeros(slots, d_inner, T + d_conv - 2, dtype=BF16, device=device)
        self.scan_state = torch.zeros(slots, d_inner, d_state, device=device)
        # the attention's layer
        self.w_qkv, self.w_attn = weight(dim, 3 * heads * head_dim), weight(heads * head_dim, dim, scale=0.3)
        self.n_q, self.n_k = (1 + weight(head_dim, scale=0.1) for _ in range(2))
        self.inv_freq = 10000.0 ** (-torch.arange(0, rot, 2, device=device).float() / rot)
        self.decay = -(2.0 ** -torch.arange(3, 3 + heads, device=device).float())
        self.attn_state = torch.zeros(slots, heads, head_dim, head_dim, device=device)
        self.norms = [1 + weight(dim, scale=0.1) for _ in range(3)]
        self.w_head = weight(dim, vocab, scale=0.5 * dim ** -0.5)
        # which token follows which: what drafts are drawn from, and a part of the target's probabilities
        self.follows = (2.0 * torch.randn(vocab, vocab, generator=gen, device=device)).softmax(-1)
        self.lengths = torch.zeros(slots, dtype=torch.int64, device=device)

    def _norm(self, x, i):
        out = torch.empty_like(x)
        cv.gated_norm(x, None, self.norms[i], out)
        return out

    def _scan_inputs(self, c):
        low = c @ self.w_low
        return low[..., :16] @ self.w_dt, low[..., 16:16 + self.d_state], low[..., 16 + self.d_state:]

    def _heads(self, x, positions):
        """Rotated q and k, and v, of [tokens, dim] rows."""
        q, k, v = (x @ self.w_qkv).unflatten(-1, (3, self.heads, self.head_dim)).unbind(1)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        cv.qk_norm_rotary(q, k, positions, self.inv_freq, qo, ko, q_weight=self.n_q, k_weight=self.n_k)
        return qo, ko, v

    def _leave(self, h, o):
        return self._norm(h + o @ self.w_attn, 2) @ self.w_head

    def prompt(self, tokens, cu_seqlens, max_len, slots):
        """Packed prompts [total]; logits of every token, states and windows left in their slots."""
        fresh = torch.zeros_like(slots)
        h = self.embed[tokens]
        x = self._norm(h, 0)
        u, z = x @ self.w_x, x @ self.w_z
        c = torch.empty_like(u)
        cv.conv_prefill(u, self.w_conv, None, self.conv_state, c, cu_seqlens, max_len=max_len, slot_idx=slots,
                        has_initial_state=fresh)
        dt, B, C = self._scan_inputs(c)
        y = torch.empty_like(c)
        cv.selective_scan_prefill(c, dt, self.A, B, C, self.scan_state, y, cu_seqlens, max_len=max_len, z=z, D=self.D,
                                  dt_bias=self.dt_bias, slot_idx=slots, has_initial_state=fresh)
        h = h + y @ self.w_scan
        lengths = (cu_seqlens[1:] - cu_seqlens[:-1]).long()
        starts = torch.repeat_interleave(cu_seqlens[:-1].long(), lengths, output_size=len(tokens))
        q, k, v = self._heads(self._norm(h, 1), torch.arange(len(tokens), device=tokens.device) - starts)
        o = torch.empty(v.shape, dtype=BF16, device=v.device)
        cv.linear_attn_prefill(q, k, v, self.decay, self.attn_state, o, cu_seqlens, max_len=max_len, slot_idx=slots,
                               has_initial_state=fresh)
        self.lengths[slots.long()] = lengths
        return self._leave(h, o.flatten(1))

    def verify(self, tokens, slots):
        """Logits behind each of [n, T] tokens, against states that stay as they are."""
        n, T = tokens.shape
        h = self.embed[tokens.clamp(min=0)]
        x = self._norm(h.flatten(0, 1), 0).view_as(h)
        u, z = x @ self.w_x, x @ self.w_z
        c = torch.empty_like(u)
        cv.conv_verify_update_dedup(u, self.w_conv, None, self.conv_state, c, self.windows, qk_channels=0, head_dim=128,
                                    slot_idx=slots)
        dt, B, C = self._scan_inputs(c)
        y = torch.empty_like(c)
        cv.selective_scan_verify(c, dt, self.A, B, C, self.scan_state, y, z=z, D=self.D, dt_bias=self.dt_bias, slot_idx=slots)
        h = (h + y @ self.w_scan).flatten(0, 1)
        positions = self.lengths[slots.long()][:, None] + torch.arange(T, device=tokens.device)
        q, k, v = (t.unflatten(0, (n, T)) for t in self._heads(self._norm(h, 1), positions.flatten()))
        o = torch.empty(v.shape, dtype=BF16, device=v.device)
        cv.linear_attn_verify(q, k, v, self.decay, self.attn_state, o, slot_idx=slots)
        self.seen = c, dt, B, k, v, slots
        return self._leave(h, o.flatten(0, 1).flatten(1)).view(n, T, -1)

    def probabilities(self, logits, tokens):
        return (logits.float() + self.follows[tokens.long()].log()).softmax(-1)

    def commit(self, num_tokens, window_index):
        c, dt, B, k, v, slots = self.seen
        cv.conv_verify_restore(self.conv_state, self.windows, window_index, layout="dedup", d_conv=self.d_conv, slot_idx=slots)
        cv.selective_scan_commit(c, dt, self.A, B, self.scan_state, num_tokens, dt_bias=self.dt_bias, slot_idx=slots)
        cv.linear_attn_commit(k, v, self.decay, self.attn_state, num_tokens, slot_idx=slots)
        self.lengths.index_add_(0, slots.long(), num_tokens.long())


def write(model, prompts, steps=4, seed=1, device="cuda"):
    """Prompts of the given lengths and `steps` steps of drafts.  Returns each row's kept tokens, the counts of
    every step, and the model's logits behind all but the last kept token by steps and by one prompt."""
    gen = torch.Generator(device).manual_seed(seed)
    n, T = len(prompts), model.T
    slots = torch.arange(n, dtype=torch.int32, device=device)
    rows = [torch.randint(0, model.vocab, (p,), generator=gen, device=device) for p in prompts]

    def packed(rows):
        cu = [0]
        for r in rows:
            cu.append(cu[-1] + len(r))
        return torch.cat(rows), torch.tensor(cu, dtype=torch.int32, device=device), max(map(len, rows))

    tokens, cu, longest = packed(rows)
    logits = model.prompt(tokens, cu, longest, slots)
    ends = cu[1:].long() - 1
    last = torch.multinomial(model.probabilities(logits[ends], tokens[ends]), 1, generator=gen)[:, 0]
    num, nxt, where = (torch.zeros(n, dtype=torch.int32, device=device) for _ in range(3))
    counts = []
    for _ in range(steps):
        chain = [last]
        for _ in range(T - 1):
            chain.append(torch.multinomial(model.follows[chain[-1]], 1, generator=gen)[:, 0])
        drafts = torch.stack(chain, 1).int()
        logits = model.verify(drafts, slots)
        cv.accept_drafts(drafts, model.probabilities(logits, drafts), torch.rand(n, T, generator=gen, device=device),
                         num, nxt, draft=model.follows[drafts[:, :-1].long()], window_index=where)
        model.commit(num, where)
        counts.append(num.tolist())                # (for the comparison below; the step itself needs no host)
        rows = [torch.cat([r, d[:c].long()]) for r, d, c in zip(rows, drafts, counts[-1])]
        stepped = logits[torch.arange(n, device=device), where.long()]
        last = nxt.long()
    tokens, cu, longest = packed(rows)
    whole = model.prompt(tokens, cu, longest, slots)[cu[1:].long() - 1]
    return rows, counts, stepped, whole


def main():
    model = SpeculativeModel()
    rows, counts, stepped, whole = write(model, [5, 300, 64, 1, 129])
    off = ((stepped.float() - whole.float()).norm() / whole.float().norm()).item()
    print("tokens kept at each step:", counts)
    print(f"last logits: off from one long prompt by {off:.4f} of their norm")


if __name__ == "__main__":
    main()
