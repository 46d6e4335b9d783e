"""Rounds of speculative decoding over a cache in 8 bits, drafts by lookup, until a few tokens are there.

    moe_round_map        pages, positions and masks of the rows
    moe_qk_rope_cache    norms and rotation; keys go to a buffer of the round's rows
    moe_cache8_append    the rows' keys and values into the paged cache, codes and scales
    moe_tree_attention8  the rows over it
    moe_verify_drafts    which drafts stand, and the token that follows
    moe_cache8_read      at the end, a request's context back in 16 bits

One attention layer with seeded random weights, the set-up that examples/verify_round.py has.  Run it on a GB300 with
the library built:  python examples/verify_round8.py
"""
from __future__ import annotations

import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from verify_round import HEAD_DIM, KV_HEADS, PAGE, Q_HEADS, VOCAB, Layer, Rows, _i32, mv  # noqa: E402

BLOCK = 8


class Layer8(Layer):
    """The layer with its cache in 8 bits."""

    def __init__(self, requests: int, fmt: int = mv.MOE_E4M3, **kw):
        super().__init__(requests, **kw)
        shape = (self.n_pages, PAGE, KV_HEADS, HEAD_DIM)
        self.codes = [torch.zeros(shape, dtype=torch.uint8, device=self.device) for _ in range(2)]
        self.scales = [torch.zeros((self.n_pages, PAGE // BLOCK, KV_HEADS), device=self.device) for _ in range(2)]
        self.format = fmt

    def cache8(self):
        k, s = self.codes[0], self.scales[0]
        return mv.make_kv_cache8(
            k.data_ptr(), self.codes[1].data_ptr(), s.data_ptr(), self.scales[1].data_ptr(), n_pages=self.n_pages,
            page_size=PAGE, block_size=BLOCK, format=self.format, page_stride=k.stride(0), slot_stride=k.stride(1),
            head_stride=k.stride(2), scale_page_stride=s.stride(0), scale_block_stride=s.stride(1), scale_head_stride=s.stride(2))

    def rows_args(self, k, v, start, ctx, rows):
        return mv.make_cache8_args(
            n_req=self.requests, n_rows=rows, kv_heads=KV_HEADS, head_dim=HEAD_DIM, dtype=mv.MOE_BF16, k=k.data_ptr(),
            v=v.data_ptr(), k_stride=k.stride(0), v_stride=v.stride(0), row_start=start.data_ptr(), ctx_len=ctx.data_ptr(),
            block_table=self.table.data_ptr(), table_width=self.width, cache=self.cache8(), dev_status=self.status.data_ptr())

    def cache_rows8(self, x, rows: Rows, ctx):
        """Rotated queries of the rows; their keys and values enter the cache."""
        qkv = (x @ self.w_qkv).view(rows.count, Q_HEADS + 2 * KV_HEADS, HEAD_DIM)
        q, k, v = qkv[:, :Q_HEADS], qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], qkv[:, Q_HEADS + KV_HEADS:]
        out = torch.empty((rows.count, Q_HEADS, HEAD_DIM), dtype=torch.bfloat16, device=self.device)
        # one page as long as the round: the rotation writes the rows' keys and values there
        staged = torch.empty((2, rows.count, KV_HEADS, HEAD_DIM), dtype=torch.bfloat16, device=self.device)
        if rows.count == 0:  # (a page has a slot at least)
            return out, staged
        page = mv.make_kv_cache(staged[0].data_ptr(), staged[1].data_ptr(), n_pages=1, page_size=rows.count, page_stride=0,
                                slot_stride=KV_HEADS * HEAD_DIM, head_stride=HEAD_DIM)
        slots = torch.arange(rows.count, dtype=torch.int32, device=self.device)
        mv.moe_qk_rope_cache(mv.make_qk_rope_args(
            n_rows=rows.count, q_heads=Q_HEADS, kv_heads=KV_HEADS, head_dim=HEAD_DIM, rot_dim=HEAD_DIM, dtype=mv.MOE_BF16,
            q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), q_stride=qkv.stride(0), k_stride=qkv.stride(0),
            v_stride=qkv.stride(0), q_out=out.data_ptr(), q_out_stride=out.stride(0), row_pos=rows.pos.data_ptr(),
            row_slot=slots.data_ptr(), cache=page, dev_status=self.status.data_ptr(), inv_freq=self.inv_freq.data_ptr(),
            q_gain=self.q_gain.data_ptr(), k_gain=self.k_gain.data_ptr()), self.stream)
        ctx = _i32(ctx, self.device)
        mv.moe_cache8_append(self.rows_args(staged[0], staged[1], rows.start, ctx, rows.count), self.stream)
        return out, staged

    def attend8(self, q, rows: Rows, ctx, widest: int):
        out = torch.empty_like(q)
        ctx = _i32(ctx, self.device)
        args = mv.make_tree_attention8_args(
            n_req=self.requests, n_rows=rows.count, max_tree=widest, q_heads=Q_HEADS, kv_heads=KV_HEADS, head_dim=HEAD_DIM,
            dtype=mv.MOE_BF16, q=q.data_ptr(), q_stride=q.stride(0), out=out.data_ptr(), out_stride=out.stride(0),
            row_start=rows.start.data_ptr(), ctx_len=ctx.data_ptr(), block_table=self.table.data_ptr(), table_width=self.width,
            cache=self.cache8(), scale=HEAD_DIM ** -0.5, dev_status=self.status.data_ptr())
        ws = torch.zeros(mv.moe_tree_attention8_workspace_bytes(args), dtype=torch.uint8, device=self.device)
        mv.moe_tree_attention8(args, ws.data_ptr(), ws.numel(), self.stream)
        return out

    def verify(self, logits, rows: Rows, tokens, uniform, noise, inv_temperature):
        accepted, follow = (torch.empty(self.requests, dtype=torch.int32, device=self.device) for _ in range(2))
        path = torch.empty(rows.count, dtype=torch.int32, device=self.device)
        args = mv.make_verify_args(
            n_req=self.requests, n_rows=rows.count, vocab=VOCAB, dtype=mv.MOE_BF16, logits=logits.data_ptr(),
            stride=logits.stride(0), row_start=rows.start.data_ptr(), tokens=tokens.data_ptr(), uniform=uniform.data_ptr(),
            noise=noise.data_ptr(), noise_stride=noise.stride(0), inv_temperature=inv_temperature, accepted=accepted.data_ptr(),
            path=path.data_ptr(), next_token=follow.data_ptr(), dev_status=self.status.data_ptr())
        ws = torch.zeros(mv.moe_verify_drafts_workspace_bytes(args), dtype=torch.uint8, device=self.device)
        mv.moe_verify_drafts(args, ws.data_ptr(), ws.numel(), self.stream)
        return accepted, path, follow

    def read(self, ctx):
        """Every request's context, keys and values in 16 bits."""
        start = _i32(np.concatenate([[0], np.cumsum(ctx)]), self.device)
        k, v = (torch.empty((sum(ctx), KV_HEADS, HEAD_DIM), dtype=torch.bfloat16, device=self.device) for _ in range(2))
        mv.moe_cache8_read(self.rows_args(k, v, start, _i32([0] * self.requests, self.device), sum(ctx)), self.stream)
        return k, v


def lookup(tokens, most):
    """What followed the last token where it stood before: drafts, none if it is new."""
    for i in range(len(tokens) - 2, -1, -1):
        if tokens[i] == tokens[-1]:
            return tokens[i + 1:i + 1 + most]
    return []


def decode(layer: Layer8, prompts, rounds, inv_temperature=1.0, drafts=4, seed=0):
    """Rounds of verification behind the prompts; returns the texts, and of each round what a test may look at."""
    dev = layer.device
    gen = torch.Generator(device=dev).manual_seed(seed)
    texts = [list(p) for p in prompts]
    ctx = [len(p) - 1 for p in texts]  # the last token's keys and values come with the first round
    prompt = layer.map_rows([0] * layer.requests, ctx)
    _, staged = layer.cache_rows8(layer.embed[_i32(sum((t[:-1] for t in texts), []), dev).long()], prompt, [0] * layer.requests)
    seen = [dict(ctx=[0] * layer.requests, staged=staged, rows=prompt)]
    for _ in range(rounds):
        chains = [[t[-1]] + lookup(t, drafts) for t in texts]
        rows = layer.map_rows(ctx, [len(c) for c in chains])
        tokens = _i32(sum(chains, []), dev)
        x = layer.embed[tokens.long()]
        q, staged = layer.cache_rows8(x, rows, ctx)
        attended = layer.attend8(q, rows, ctx, max(len(c) for c in chains))
        logits = (x + attended.view(rows.count, -1) @ layer.w_out) @ layer.w_vocab
        uniform = torch.rand(rows.count, generator=gen, device=dev)
        noise = torch.empty((layer.requests, VOCAB), device=dev).exponential_(generator=gen)
        accepted, path, follow = layer.verify(logits, rows, tokens, uniform, noise, inv_temperature)
        seen.append(dict(ctx=list(ctx), chains=chains, rows=rows, q=q, staged=staged, attended=attended, logits=logits,
                         uniform=uniform, noise=noise, accepted=accepted, path=path, follow=follow))
        for b, (n, token) in enumerate(zip(accepted.tolist(), follow.tolist())):
            texts[b] += chains[b][1:1 + n] + [token]
            ctx[b] += 1 + n  # the rows that stand; the others' places are taken by the next round's
    return texts, ctx, seen


def main():
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (30, 25)]
    for _ in range(2):  # the second time behind the first's texts, with the same token last: the drafts are what followed it
        layer = Layer8(requests=2)
        texts, ctx, seen = decode(layer, prompts, rounds=6, inv_temperature=math.inf)
        k, _ = layer.read(ctx)
        assert int(layer.status.item()) == 0 and bool(torch.isfinite(k).all())
        for b, (p, t) in enumerate(zip(prompts, texts)):
            stood = [int(s["accepted"][b]) for s in seen[1:]]
            print(f"request {b}: {len(t) - len(p)} tokens in {len(stood)} rounds, drafts that stood {stood}: {t[len(p):]}")
        layer.close()
        prompts = [t + [p[-1]] for p, t in zip(prompts, texts)]


if __name__ == "__main__":
    main()
