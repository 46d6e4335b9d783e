"""One verify round of a decoder layer, from the requests' lengths to the accepted drafts.

Two phases share the calls: the prompts' keys and values enter the paged cache, then every
request brings a tree of drafted tokens and one layer runs over all of them:

    moe_round_map        pages, cache slots, positions and tree masks of the rows
    moe_qk_rope_cache    norms and rotation of queries and keys, keys and values cached
    moe_tree_attention   the drafted rows over the cached context and their ancestors
    moe_decode_layer     the expert layer over the same rows
    moe_token_logprobs   the drafted tokens under the logits

The projections are plain torch matrix products with seeded random weights.  Run it on a
GB300 with the library built:  python examples/verify_round.py
"""
from __future__ import annotations

import os
import sys
from typing import NamedTuple

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import spec_verify_layer_gb300 as mv  # noqa: E402
import syngen  # noqa: E402
from spec_verify_layer_gb300.weights import upload_layer, workspace  # noqa: E402

Q_HEADS, KV_HEADS, HEAD_DIM, PAGE, VOCAB, TOP = 8, 2, 64, 16, 1000, 4


def _i32(values, device):
    return torch.tensor(np.asarray(values, np.int64), dtype=torch.int32, device=device)


class Rows(NamedTuple):
    """What moe_round_map says about the rows of a phase."""
    start: torch.Tensor
    pos: torch.Tensor
    slot: torch.Tensor
    mask: torch.Tensor | None
    count: int


class Layer:
    """A decoder layer of a small shape with a paged cache, its free pages and its descriptors' buffers."""

    def __init__(self, requests: int, pages: int = 64, width: int = 16, seed: int = 0, device="cuda:0"):
        self.device = torch.device(device)
        self.cfg = syngen.CONFIGS["tiny"].with_(rows=16)
        self.hidden, self.requests, self.width = self.cfg.hidden, requests, width
        gen = torch.Generator(device=self.device).manual_seed(seed)
        rand = lambda *n: (torch.randn(n, generator=gen, device=self.device) / n[0] ** 0.5).bfloat16()  # noqa: E731
        self.w_qkv = rand(self.hidden, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM)
        self.w_out, self.w_vocab = rand(Q_HEADS * HEAD_DIM, self.hidden), rand(self.hidden, VOCAB)
        self.embed = torch.randn((VOCAB, self.hidden), generator=gen, device=self.device).bfloat16()
        self.q_gain = (1 + 0.1 * torch.randn(HEAD_DIM, generator=gen, device=self.device)).bfloat16()
        self.k_gain = (1 + 0.1 * torch.randn(HEAD_DIM, generator=gen, device=self.device)).bfloat16()
        self.inv_freq = 1e4 ** (-torch.arange(0, HEAD_DIM, 2, device=self.device, dtype=torch.float64) / HEAD_DIM)
        shape = (pages, PAGE, KV_HEADS, HEAD_DIM)
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=torch.bfloat16, device=self.device) for _ in range(2))
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=self.device)
        self.held = torch.zeros(requests, dtype=torch.int32, device=self.device)
        self.free, self.n_pages = list(range(pages)), pages
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.dims = mv.make_dims(self.hidden, self.cfg.experts, self.cfg.top_k, self.cfg.inter, 16)
        self.experts = upload_layer(self.dims, syngen.router(self.cfg, 0), lambda e: syngen.expert(self.cfg, 0, e),
                                    self.device)
        self.handle = mv.moe_create(self.dims, self.device.index or 0)

    def close(self):
        mv.moe_destroy(self.handle)

    @property
    def stream(self) -> int:
        return torch.cuda.current_stream(self.device).cuda_stream

    def _cache(self):
        k = self.k_cache
        return mv.make_kv_cache(k.data_ptr(), self.v_cache.data_ptr(), n_pages=self.n_pages, page_size=PAGE,
                                page_stride=k.stride(0), slot_stride=k.stride(1), head_stride=k.stride(2))

    def map_rows(self, ctx, new, parents=None) -> Rows:
        """Pages and slots for `new` rows behind `ctx` cached positions of each request."""
        n, dev = int(sum(new)), self.device
        ctx_d, new_d, free = _i32(ctx, dev), _i32(new, dev), _i32(self.free, dev)
        up = None if parents is None else _i32(parents, dev)
        start, pages, taken = (torch.empty(m, dtype=torch.int32, device=dev) for m in (self.requests + 1, self.requests, 1))
        req, pos, slot = (torch.empty(n, dtype=torch.int32, device=dev) for _ in range(3))
        mask = None if parents is None else torch.empty(n, dtype=torch.int64, device=dev)
        mv.moe_round_map(mv.make_map_args(
            n_req=self.requests, n_rows=n, page_size=PAGE, n_pages=self.n_pages, table_width=self.width,
            n_free=len(self.free), ctx_len=ctx_d.data_ptr(), new_len=new_d.data_ptr(), pages_held=self.held.data_ptr(),
            free_pages=free.data_ptr(), parents=0 if up is None else up.data_ptr(), block_table=self.table.data_ptr(),
            row_start=start.data_ptr(), pages=pages.data_ptr(), n_taken=taken.data_ptr(), row_req=req.data_ptr(),
            row_pos=pos.data_ptr(), row_slot=slot.data_ptr(), tree_mask=0 if mask is None else mask.data_ptr(),
            dev_status=self.status.data_ptr()), self.stream)
        self.held = pages
        self.free = self.free[int(taken.item()):]  # the pool's book-keeping is the program's
        return Rows(start, pos, slot, mask, n)

    def cache_rows(self, x, rows: Rows):
        """Rotated queries of the rows; their keys and values enter the cache."""
        qkv = (x @ self.w_qkv).view(rows.count, Q_HEADS + 2 * KV_HEADS, HEAD_DIM)
        q, k, v = qkv[:, :Q_HEADS], qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], qkv[:, Q_HEADS + KV_HEADS:]
        out = torch.empty((rows.count, Q_HEADS, HEAD_DIM), dtype=torch.bfloat16, device=self.device)
        mv.moe_qk_rope_cache(mv.make_qk_rope_args(
            n_rows=rows.count, q_heads=Q_HEADS, kv_heads=KV_HEADS, head_dim=HEAD_DIM, rot_dim=HEAD_DIM,
            dtype=mv.MOE_BF16, q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), q_stride=qkv.stride(0),
            k_stride=qkv.stride(0), v_stride=qkv.stride(0), q_out=out.data_ptr(), q_out_stride=out.stride(0),
            row_pos=rows.pos.data_ptr(), row_slot=rows.slot.data_ptr(), cache=self._cache(),
            dev_status=self.status.data_ptr(), inv_freq=self.inv_freq.data_ptr(), q_gain=self.q_gain.data_ptr(),
            k_gain=self.k_gain.data_ptr()), self.stream)
        return out, qkv

    def attend(self, q, rows: Rows, ctx, widest: int):
        out = torch.empty_like(q)
        ctx_d = _i32(ctx, self.device)
        args = mv.make_tree_attention_args(
            n_req=self.requests, n_rows=rows.count, max_tree=widest, q_heads=Q_HEADS, kv_heads=KV_HEADS,
            head_dim=HEAD_DIM, dtype=mv.MOE_BF16, q=q.data_ptr(), q_stride=q.stride(0), out=out.data_ptr(),
            out_stride=out.stride(0), row_start=rows.start.data_ptr(), ctx_len=ctx_d.data_ptr(),
            block_table=self.table.data_ptr(), table_width=self.width, cache=self._cache(), scale=HEAD_DIM ** -0.5,
            dev_status=self.status.data_ptr(), tree_mask=rows.mask.data_ptr())
        ws = torch.zeros(mv.moe_tree_attention_workspace_bytes(args), dtype=torch.uint8, device=self.device)
        mv.moe_tree_attention(args, ws.data_ptr(), ws.numel(), self.stream)
        return out

    def expert_layer(self, x):
        out = torch.empty(x.shape, dtype=torch.float32, device=self.device)
        ws = workspace(self.dims, x.shape[0], self.device)
        mv.moe_decode_layer(self.handle, self.experts.w, x.view(torch.int16).data_ptr(), x.shape[0], out.data_ptr(),
                            ws.data_ptr(), ws.numel(), self.stream)
        return out

    def score(self, logits, tokens):
        """Log probability, entropy, rank and the first alternatives of a token under each row's logits."""
        n = logits.shape[0]
        logp, entropy = (torch.empty(n, device=self.device) for _ in range(2))
        rank, top_ids = (torch.empty(m, dtype=torch.int32, device=self.device) for m in ((n,), (n, TOP)))
        top_logp = torch.empty((n, TOP), device=self.device)
        args = mv.make_logprob_args(
            n_rows=n, vocab=VOCAB, dtype=mv.MOE_BF16, logits=logits.data_ptr(), stride=logits.stride(0),
            dev_status=self.status.data_ptr(), tokens=tokens.data_ptr(), top_k=TOP, logp=logp.data_ptr(),
            entropy=entropy.data_ptr(), rank=rank.data_ptr(), top_ids=top_ids.data_ptr(), top_logp=top_logp.data_ptr())
        ws = torch.zeros(mv.moe_token_logprobs_workspace_bytes(args), dtype=torch.uint8, device=self.device)
        mv.moe_token_logprobs(args, ws.data_ptr(), ws.numel(), self.stream)
        return logp, entropy, rank, top_ids, top_logp


def verify_round(layer: Layer, prompts, drafts, parents):
    """prompts, drafts: token lists of each request; parents: each draft's parent in its tree (-1: the prompt's
    last token).  Returns everything a caller or a test may want to look at."""
    dev = layer.device
    ctx, none = [len(p) for p in prompts], [0] * layer.requests
    prompt = layer.map_rows(none, ctx)
    _, prompt_qkv = layer.cache_rows(layer.embed[_i32(sum(prompts, []), dev).long()], prompt)

    tokens = _i32(sum(drafts, []), dev)
    rows = layer.map_rows(ctx, [len(d) for d in drafts], sum(parents, []))
    x = layer.embed[tokens.long()]
    q, qkv = layer.cache_rows(x, rows)
    attended = layer.attend(q, rows, ctx, max(len(d) for d in drafts))
    h = (x.float() + (attended.view(rows.count, -1) @ layer.w_out).float()).bfloat16()
    h = (h.float() + layer.expert_layer(h)).bfloat16()
    logits = h @ layer.w_vocab
    # the row's children are its continuation: score each draft under its parent's logits (roots are left out)
    base = np.repeat(np.cumsum([0] + [len(d) for d in drafts])[:-1], [len(d) for d in drafts])
    up = np.asarray(sum(parents, []))
    child = np.nonzero(up >= 0)[0]
    under = torch.from_numpy((base + up)[child]).to(dev)
    scores = layer.score(logits[under].contiguous(), tokens[torch.from_numpy(child).to(dev)].contiguous())
    return dict(prompt=prompt, prompt_qkv=prompt_qkv, rows=rows, qkv=qkv, q=q, attended=attended, logits=logits,
                child=child, under=under, tokens=tokens, scores=scores, status=int(layer.status.item()))


def main():
    layer = Layer(requests=2)
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (41, 16)]
    drafts = [rng.integers(0, VOCAB, n).tolist() for n in (6, 4)]
    parents = [[-1, 0, 1, 1, 0, 4], [-1, 0, 1, 2]]
    r = verify_round(layer, prompts, drafts, parents)
    assert r["status"] == 0
    logp, entropy, rank, top_ids, _ = (t.cpu().numpy() for t in r["scores"])
    for i, c in enumerate(r["child"]):
        print(f"draft {c}: token {int(r['tokens'][c])} log p {logp[i]:.3f} rank {rank[i]} entropy {entropy[i]:.3f} "
              f"instead {top_ids[i].tolist()}")
    layer.close()


if __name__ == "__main__":
    main()
