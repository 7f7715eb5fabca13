"""A hybrid linear-attention layer on the framework's kernels, from a prompt through speculative
decoding:

    prompt   conv_prefill -> conv_qk_l2norm -> linear_attn_prefill -> gated_norm -> residual_norm
    verify   conv_verify_update_dedup -> linear_attn_verify -> gated_norm -> residual_norm
    commit   conv_verify_restore (the conv window) and linear_attn_commit (the state)

The projections around them are torch products.  Run as a program it serves random prompts and
drafts, accepts some of each, and compares what the layer says about the last drafts with one
long prompt over the same tokens:

    python examples/hybrid_layer.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_conv1d_verify_amd as cv  # noqa: E402

BF16 = torch.bfloat16


class HybridLayer:
    """One layer's weights and its pools: conv windows, rollback rows and attention states."""

    def __init__(self, dim=512, q_heads=4, v_heads=8, dk=64, dv=64, drafts=6, slots=8, d_conv=4,
                 device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)

        def weight(*shape, scale):
            return (scale * torch.randn(*shape, generator=gen, device=device)).to(BF16)

        self.q_heads, self.v_heads, self.dk, self.dv, self.drafts = q_heads, v_heads, dk, dv, drafts
        self.qk, self.d_inner = 2 * q_heads * dk, 2 * q_heads * dk + v_heads * dv
        self.w_in = weight(dim, self.d_inner, scale=dim ** -0.5)
        self.w_gate = weight(dim, v_heads * dv, scale=dim ** -0.5)
        self.w_decay = weight(dim, v_heads, scale=dim ** -0.5)
        self.rate = 1 + 7 * torch.rand(v_heads, generator=gen, device=device)
        self.w_conv = weight(self.d_inner, d_conv, scale=0.5)
        self.w_out = weight(v_heads * dv, dim, scale=(v_heads * dv) ** -0.5)
        self.n_head, self.n_post, self.n_pre = (1 + weight(n, scale=0.1) for n in (dv, dim, dim))
        self.conv_state = torch.zeros(slots, self.d_inner, d_conv - 1, dtype=BF16, device=device)
        self.rows = torch.zeros(slots, self.d_inner, drafts + d_conv - 2, dtype=BF16, device=device)
        self.state = torch.zeros(slots, v_heads, dk, dv, device=device)
        self.d_conv = d_conv

    def _decays(self, x):
        return -self.rate * torch.nn.functional.softplus((x @ self.w_decay).float() - 3)

    def _heads(self, y):
        """q, k and v as views of the conv's output rows."""
        a = self.q_heads * self.dk
        return (y[..., :a].unflatten(-1, (self.q_heads, self.dk)),
                y[..., a:2 * a].unflatten(-1, (self.q_heads, self.dk)),
                y[..., 2 * a:].unflatten(-1, (self.v_heads, self.dv)))

    def _leave(self, o, x, residual):
        """The attention's output to the next block: its input; `residual` is updated in place."""
        z = (x @ self.w_gate).view(-1, self.v_heads, self.dv)
        o = o.reshape(-1, self.v_heads, self.dv)
        cv.gated_norm(o, z, self.n_head, o)
        y = o.flatten(1) @ self.w_out
        out = torch.empty_like(y)
        cv.residual_norm(y, residual, self.n_pre, out, post_weight=self.n_post)
        return out

    def prompt(self, x, residual, cu_seqlens, max_len, slots):
        """Packed prompts [total, dim]; their windows and states are left in their slots."""
        fresh = torch.zeros_like(slots)
        y = x @ self.w_in
        c = torch.empty_like(y)
        cv.conv_prefill(y, self.w_conv, None, self.conv_state, c, cu_seqlens, max_len=max_len,
                        slot_idx=slots, has_initial_state=fresh)
        cv.conv_qk_l2norm(c, qk_channels=self.qk, head_dim=self.dk)
        q, k, v = self._heads(c)
        o = torch.empty(v.shape, dtype=BF16, device=x.device)
        cv.linear_attn_prefill(q, k, v, self._decays(x), self.state, o, cu_seqlens,
                               max_len=max_len, slot_idx=slots, has_initial_state=fresh)
        return self._leave(o, x, residual)

    def verify(self, x, residual, slots):
        """Draft tokens [n, drafts, dim] against the states, which stay as they are."""
        y = x @ self.w_in
        c = torch.empty_like(y)
        cv.conv_verify_update_dedup(y, self.w_conv, None, self.conv_state, c, self.rows,
                                    qk_channels=self.qk, head_dim=self.dk, slot_idx=slots)
        q, k, v = self._heads(c)
        g = self._decays(x)
        self.seen = k, v, g, slots
        o = torch.empty(v.shape, dtype=BF16, device=x.device)
        cv.linear_attn_verify(q, k, v, g, self.state, o, slot_idx=slots)
        return self._leave(o, x.flatten(0, 1), residual.flatten(0, 1)).view(x.shape)

    def commit(self, accepted):
        """The first accepted[i] (1 or more) of row i's drafts are kept."""
        k, v, g, slots = self.seen
        cv.conv_verify_restore(self.conv_state, self.rows, accepted - 1, layout="dedup",
                               d_conv=self.d_conv, slot_idx=slots)
        cv.linear_attn_commit(k, v, g, self.state, accepted, slot_idx=slots)


def serve(layer, prompts, rounds=3, seed=1, device="cuda"):
    """Prompts of the given lengths, then rounds of drafts of which some are accepted.  Returns
    the layer's outputs for the last drafts, and one prompt's over each row's tokens."""
    gen = torch.Generator(device).manual_seed(seed)
    n, dim, T = len(prompts), layer.w_in.shape[0], layer.drafts

    def tokens(*shape):
        return torch.randn(*shape, dim, generator=gen, device=device).to(BF16)

    slots = torch.arange(n, dtype=torch.int32, device=device)
    x = tokens(sum(prompts))
    kept = list(x.split(prompts))
    cu = torch.tensor([0, *torch.tensor(prompts).cumsum(0).tolist()], dtype=torch.int32, device=device)
    layer.prompt(x, x.clone(), cu, max(prompts), slots)
    for r in range(rounds):
        d = tokens(n, T)
        out = layer.verify(d, d.clone(), slots)
        if r + 1 < rounds:
            accepted = torch.randint(1, T + 1, (n,), generator=gen, device=device, dtype=torch.int32)
            layer.commit(accepted)
            kept = [torch.cat([a, b[:c]]) for a, b, c in zip(kept, d, accepted.tolist())]
    whole = [torch.cat([a, b]) for a, b in zip(kept, d)]
    lengths = [len(w) for w in whole]
    x = torch.cat(whole)
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=device)
    want = layer.prompt(x, x.clone(), cu, max(lengths), slots)
    return out, torch.stack([w[-T:] for w in want.split(lengths)])


def main():
    layer = HybridLayer()
    out, want = serve(layer, [5, 300, 64, 1, 129])
    off = ((out.float() - want.float()).norm() / want.float().norm()).item()
    print(f"last drafts {tuple(out.shape)}: off from one long prompt by {off:.4f} of their norm")


if __name__ == "__main__":
    main()
