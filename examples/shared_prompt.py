"""Several continuations of one prompt with caches of bounded size.

The toy target of target_cycle.py, whose B sequences begin with the same pages:

  prompt   its keys and values are appended once, to pages that every page
           table begins with; each sequence draws its own first token
  cycle    a draft of K tokens; dflash_kv_append_axes with the tokens'
           positions (a slot is not a position once a cache was evicted),
           dflash_shared_attn (the prompt's pages are read once for all
           sequences), logits, dflash_sample and dflash_verify;
           dflash_logprobs of the emitted tokens with their alternatives;
           dflash_attn_mass adds the weights that the accepted queries gave
           to the sequences' own tokens; dflash_kv_evict bounds the caches

Run on a GB300:  python examples/shared_prompt.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from target_cycle import Filters, ToyTarget, dv, stand_in_draft  # noqa: E402


class SharedTarget(ToyTarget):
    """A ToyTarget whose sequences begin with the first `shared` tokens of
    sequence 0 (whole pages); what tokens gather of attention is kept in mass."""

    def __init__(self, B, K, shared, budget, recent, **sizes):
        super().__init__(B, K, **sizes)
        page = self.k_codes.shape[2]
        if shared % page:
            raise ValueError("shared must be whole pages")
        self.shared, self.budget, self.recent = shared, budget, recent
        self.table[:, :shared // page] = self.table[:1, :shared // page]
        dev = self.table.device
        slots = self.table.shape[1] * page
        f32 = dict(dtype=torch.float32, device=dev)
        self.mass = torch.zeros(B, self.Hkv, slots, **f32)
        self.mass_out = torch.zeros_like(self.mass)
        self.slots = torch.full((B,), shared, dtype=torch.int32, device=dev)
        self.new_len = torch.empty_like(self.slots)
        self.evict_ws = torch.empty(dv.dflash_kv_evict_workspace_bytes(
            B, self.Hkv, page, budget), dtype=torch.uint8, device=dev)
        self.pool = (self.k_codes, self.v_codes, self.k_scale, self.v_scale)

    def prompt_logits(self, prompt):
        """Logits [V] after the prompt (its `shared` tokens), whose keys and
        values go to the pages that all sequences begin with."""
        n = prompt.numel()
        x = self.emb[prompt.long()]
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        q, k, v = (x @ self.w_qkv.T).split([Hq * D, Hkv * D, Hkv * D], 1)
        q_rot = torch.empty(1, n, Hq, D, dtype=x.dtype, device=x.device)
        length = torch.zeros(1, dtype=torch.int32, device=x.device)
        dv.dflash_kv_append(q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)),
                            v.unflatten(1, (Hkv, D)), self.cos, self.sin,
                            torch.zeros_like(length), None, self.table[:1],
                            *self.pool, q_rot, length)
        out = torch.empty_like(q_rot)
        ws = torch.empty(dv.dflash_paged_attn_workspace_bytes(
            1, n, Hq, Hkv, D), dtype=torch.uint8, device=x.device)
        dv.dflash_paged_attn(q_rot, *self.pool, self.table[:1], length, None,
                             D ** -0.5, out, None, ws)
        y = x[-1] + out[0, -1].view(-1)
        return self.sharp * (y @ self.w_out.T).float()

    def logits(self, tokens, positions):
        """Logits [B, Q, V] fp32 of tokens [B, Q] at `positions` [B] and on,
        appended from slot self.slots on; keeps what count() needs."""
        B, Q = tokens.shape
        x = self.emb[tokens.long()].view(B * Q, -1)
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        q, k, v = (x @ self.w_qkv.T).split([Hq * D, Hkv * D, Hkv * D], 1)
        self.q_rot = torch.empty(B, Q, Hq, D, dtype=x.dtype, device=x.device)
        at = (positions[:, None] + torch.arange(
            Q, dtype=torch.int32, device=x.device)).view(1, B * Q)
        dv.dflash_kv_append_axes(
            q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)),
            v.unflatten(1, (Hkv, D)), self.cos, self.sin, at, None,
            self.slots, None, self.table, *self.pool, self.q_rot, self.kv_len)
        out = torch.empty_like(self.q_rot)
        self.lse = torch.empty(B, Q, Hq, device=x.device)
        if Q not in self._ws:
            self._ws[Q] = torch.empty(dv.dflash_shared_attn_workspace_bytes(
                B, Q, Hq, Hkv, D), dtype=torch.uint8, device=x.device)
        dv.dflash_shared_attn(self.q_rot, *self.pool, self.table, self.kv_len,
                              None, self.shared, D ** -0.5, out, self.lse,
                              self._ws[Q])
        y = x + out.view(B * Q, -1)
        return (self.sharp * (y @ self.w_out.T).float()).view(B, Q, self.V)

    def count(self, n):
        """The first n[b] + 1 tokens of the last block were accepted: their
        queries' weights are counted, the caches cut to the budget."""
        new = n + 1
        kv_len = self.slots + new
        dv.dflash_attn_mass(self.q_rot, self.k_codes, self.k_scale,
                            self.table, kv_len, new, self.lse, self.slots,
                            self.shared, self.D ** -0.5, 1.0, self.mass)
        dv.dflash_kv_evict(self.mass, *self.pool, self.table, kv_len,
                           self.budget, self.shared, self.recent,
                           self.mass_out, self.new_len, None, self.evict_ws)
        self.mass, self.mass_out = self.mass_out, self.mass
        self.slots, self.new_len = self.new_len, self.slots


def generate(target, prompt, anchor, cycles, filters, seed=0, top=4):
    """From the prompt and each sequence's first token.  Returns the committed
    tokens, their counts, and for every cycle (n, log probabilities, ranks,
    alternatives' log probabilities and ids) of the emitted tokens."""
    B, K, V = target.B, target.K, target.V
    dev = prompt.device
    i32 = dict(dtype=torch.int32, device=dev)
    gen = torch.Generator(device=dev).manual_seed(seed)
    capacity = 1 + cycles * (K + 1)
    tokens = torch.full((B, capacity), -1, **i32)
    tokens[:, 0] = anchor
    anchor = anchor.clone()
    length = torch.ones(B, **i32)
    stats = torch.zeros(dv.COMMIT_STATS, dtype=torch.int64, device=dev)
    n = torch.empty(B, **i32)
    out_tok = torch.empty(B, K + 1, **i32)
    ws = torch.empty(dv.dflash_workspace_bytes(1, B, K, 0, V),
                     dtype=torch.uint8, device=dev)
    R = B * (K + 1)
    filtered = torch.empty(R, V, device=dev)
    said = []
    for c in range(cycles):
        draft, topi, q = stand_in_draft(target, anchor, K)
        block = torch.cat([anchor[:, None], draft], 1)
        l = target.logits(block, prompt.numel() + length - 1).view(R, V)
        filters.sample(l, torch.rand(R, generator=gen, device=dev), filtered)
        dv.dflash_verify(filtered.view(B, K + 1, V), draft, topi, q,
                         filters.T, seed, c, n, out_tok, ws)
        emitted = torch.where(
            torch.arange(K + 1, device=dev) <= n[:, None], out_tok, -1)
        logprob, best = torch.empty(R, device=dev), torch.empty(
            R, top, device=dev)
        rank, ids = torch.empty(R, **i32), torch.empty(R, top, **i32)
        dv.dflash_logprobs(l, None, emitted.view(R), logprob, rank, None, None,
                           best, ids)
        target.count(n)
        said.append((n.clone(), logprob.view(B, K + 1), rank.view(B, K + 1),
                     best, ids))
        dv.dflash_commit(n, out_tok, anchor, tokens, length, stats)
    dv.dflash_check()
    return tokens, length, said


def first_tokens(target, prompt, filters, seed=0):
    """The prompt into the shared pages, and a token for every sequence."""
    l = target.prompt_logits(prompt).repeat(target.B, 1)
    gen = torch.Generator(device=l.device).manual_seed(seed)
    return filters.sample(l, torch.rand(target.B, generator=gen,
                                        device=l.device))


def main():
    B, K, cycles = 6, 4, 24
    g = torch.Generator().manual_seed(1)
    filters = Filters(T=1.0, top_k=20, top_p=0.9)
    for budget in (400, 112):
        target = SharedTarget(B, K, shared=64, budget=budget, recent=16)
        prompt = torch.randint(0, target.V, (64,), generator=g,
                               dtype=torch.int32).cuda()
        anchor = first_tokens(target, prompt, filters)
        tokens, length, said = generate(target, prompt, anchor, cycles,
                                        filters)
        surprise = -sum(lp.sum() for _, lp, *_ in said) / (length - 1).sum()
        print(f"budget {budget}: {int(length.sum())} tokens, at most "
              f"{int(target.slots.max())} cached each, {float(surprise):.2f} "
              f"nats a token; first: {tokens[0, :8].tolist()}")


if __name__ == "__main__":
    main()
