"""A target model's side of the draft-verify loop, end to end.

A toy target (one attention layer with rotated positions, random weights)
generates tokens with the library's calls:

  prompt   dflash_kv_append of the whole prompt, dflash_paged_attn over it,
           logits of the last token, dflash_sample draws the first token
  cycle    a draft of K tokens with its candidates and probabilities;
           dflash_kv_append of the K + 1 tokens at the committed length (the
           tokens the last verify rejected are overwritten),
           dflash_paged_attn, logits, dflash_sample filters them,
           dflash_verify accepts and draws, dflash_commit hands over

The drafts come from a stand-in that only knows the last token (this example
is about the target; DraftVerify is the library's own drafter).  Run on a
GB300:  python examples/target_cycle.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_drafter_verify_gb300 as dv  # noqa: E402

C = dv.C


class ToyTarget:
    """Weights and buffers of B sequences: embedding, one attention layer,
    output head; the paged cache with its table."""

    def __init__(self, B, K, V=512, Hq=8, Hkv=2, D=64, page=16, tokens=512,
                 seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.B, self.K, self.V = B, K, V
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        H = Hq * D
        bf = torch.bfloat16

        def weights(*shape):
            return (torch.randn(*shape, generator=g) /
                    shape[-1] ** 0.5).to(bf).to(device)

        self.emb = torch.randn(V, H, generator=g).to(bf).to(device)
        self.w_qkv = weights((Hq + 2 * Hkv) * D, H)
        self.w_out = weights(V, H)
        self.sharp = 6.0                       # spread of the logits
        per = tokens // page
        order = torch.randperm(B * per, generator=g).to(torch.int32)
        self.table = order.view(B, per).to(device)
        shape = (B * per, Hkv, page, D)
        self.k_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.k_scale = torch.zeros(shape[:2], device=device)
        self.v_scale = torch.zeros(shape[:2], device=device)
        f = 10000.0 ** (-torch.arange(0, D, 2) / D)
        a = torch.arange(tokens)[:, None] * f
        self.cos, self.sin = a.cos().to(device), a.sin().to(device)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=device)
        self._ws = {}

    def logits(self, tokens, pos, n_new=None):
        """Logits [B, Q, V] fp32 of tokens [B, Q] at positions pos.. (their
        keys and values appended on the way)."""
        B, Q = tokens.shape
        x = self.emb[tokens.long()].view(B * Q, -1)
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        q, k, v = (x @ self.w_qkv.T).split([Hq * D, Hkv * D, Hkv * D], 1)
        q_rot = torch.empty(B, Q, Hq, D, dtype=x.dtype, device=x.device)
        dv.dflash_kv_append(q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)),
                            v.unflatten(1, (Hkv, D)), self.cos, self.sin, pos,
                            n_new, self.table, self.k_codes, self.v_codes,
                            self.k_scale, self.v_scale, q_rot, self.kv_len)
        out = torch.empty_like(q_rot)
        if Q not in self._ws:
            self._ws[Q] = torch.empty(dv.dflash_paged_attn_workspace_bytes(
                B, Q, Hq, Hkv, D), dtype=torch.uint8, device=x.device)
        dv.dflash_paged_attn(q_rot, self.k_codes, self.v_codes, self.k_scale,
                             self.v_scale, self.table, self.kv_len, n_new,
                             D ** -0.5, out, None, self._ws[Q])
        y = x + out.view(B * Q, -1)
        return (self.sharp * (y @ self.w_out.T).float()).view(B, Q, self.V)


class Filters:
    """One temperature, top-k, top-p and min-p for every row."""

    def __init__(self, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
        self.T, self.top_k, self.top_p, self.min_p = T, top_k, top_p, min_p

    def sample(self, logits, u, filtered=None):
        R, V = logits.shape
        dev = logits.device
        full = lambda v, t: torch.full((R,), v, dtype=t, device=dev)  # noqa: E731
        token = torch.empty(R, dtype=torch.int32, device=dev)
        ws = torch.empty(dv.dflash_sample_workspace_bytes(R, V),
                         dtype=torch.uint8, device=dev)
        dv.dflash_sample(logits, full(self.T, torch.float32),
                         full(self.top_k, torch.int32),
                         full(self.top_p, torch.float32),
                         full(self.min_p, torch.float32), u, token, None,
                         filtered, ws)
        return token


def stand_in_draft(target, anchor, K):
    """K drafted tokens from the embedding and the output head alone, greedy;
    candidates 0..15 hold the draft first, q is one-hot."""
    B = anchor.numel()
    draft = torch.empty(B, K, dtype=torch.int32, device=anchor.device)
    topi = torch.empty(B, K, C, dtype=torch.int32, device=anchor.device)
    last = anchor
    for t in range(K):
        l = target.emb[last.long()] @ target.w_out.T
        topi[:, t] = l.float().topk(C, dim=1).indices.to(torch.int32)
        last = topi[:, t, 0].contiguous()
        draft[:, t] = last
    q = torch.zeros(B, K, C, device=anchor.device)
    q[..., 0] = 1.0
    return draft, topi, q


def generate(target, prompt, lengths, cycles, filters, seed=0):
    """prompt [B, P] (lengths [B] tokens of each are real).  Returns the
    committed tokens [B, capacity], their counts and dflash_commit's
    statistics."""
    B, K, V = target.B, target.K, target.V
    dev = prompt.device
    i32 = dict(dtype=torch.int32, device=dev)
    gen = torch.Generator(device=dev).manual_seed(seed)
    zero = torch.zeros(B, **i32)
    l = target.logits(prompt, zero, lengths)
    rows = torch.arange(B, device=dev)
    first = l[rows, lengths.long() - 1].contiguous()
    anchor = filters.sample(first, torch.rand(B, generator=gen, device=dev))
    capacity = 1 + cycles * (K + 1)
    tokens = torch.full((B, capacity), -1, **i32)
    tokens[:, 0] = anchor
    length = torch.ones(B, **i32)
    stats = torch.zeros(dv.COMMIT_STATS, dtype=torch.int64, device=dev)
    n = torch.empty(B, **i32)
    out_tok = torch.empty(B, K + 1, **i32)
    ws = torch.empty(dv.dflash_workspace_bytes(1, B, K, 0, V),
                     dtype=torch.uint8, device=dev)
    filtered = torch.empty(B * (K + 1), V, device=dev)
    for c in range(cycles):
        draft, topi, q = stand_in_draft(target, anchor, K)
        block = torch.cat([anchor[:, None], draft], 1)
        # the anchor's keys are not in the cache yet: it goes first
        pos = lengths + length - 1
        l = target.logits(block, pos).view(B * (K + 1), V)
        filters.sample(l, torch.rand(B * (K + 1), generator=gen, device=dev),
                       filtered)
        dv.dflash_verify(filtered.view(B, K + 1, V), draft, topi, q,
                         filters.T, seed, c, n, out_tok, ws)
        dv.dflash_commit(n, out_tok, anchor, tokens, length, stats)
    dv.dflash_check()
    return tokens, length, stats


def main():
    B, K, cycles = 4, 4, 24
    target = ToyTarget(B, K)
    g = torch.Generator().manual_seed(1)
    prompt = torch.randint(0, target.V, (B, 40), generator=g,
                           dtype=torch.int32).cuda()
    lengths = torch.tensor([40, 17, 1, 33], dtype=torch.int32, device="cuda")
    for f in (Filters(T=0.0), Filters(T=1.0, top_k=20, top_p=0.9)):
        tokens, length, stats = generate(target, prompt, lengths, cycles, f)
        s = stats.tolist()
        print(f"T={f.T} top_k={f.top_k} top_p={f.top_p}: "
              f"{s[2]} tokens in {s[1]} verification passes, mean accepted "
              f"{s[0] / s[1]:.2f}; first: {tokens[0, :8].tolist()}")


if __name__ == "__main__":
    main()
