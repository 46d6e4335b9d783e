"""Plain implementations in 64 bits of the attention-side operators, and set-up shared by their tests."""
from __future__ import annotations

import math

import numpy as np
import torch

import spec_verify_layer_gb300 as mv

DEV = "cuda"
DT = {"bf16": (torch.bfloat16, mv.MOE_BF16), "f16": (torch.float16, mv.MOE_F16), "f32": (torch.float32, mv.MOE_F32)}


def at(t):
    return 0 if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def i32(values):
    return torch.tensor(np.asarray(values, np.int64), dtype=torch.int32, device=DEV)


# ---- page and slot map ---------------------------------------------------------------

class MapCase:
    """Lengths of a round and what a pool of pages looks like for them."""

    def __init__(self, seed, ctx, new, page, *, extra=0, tree=False, held=True, pad=0, spare=5, width=None):
        rng = np.random.default_rng(seed)
        self.page, self.pad = page, pad
        self.ctx, self.new = np.asarray(ctx, np.int64), np.asarray(new, np.int64)
        first = -(-np.maximum(self.ctx, 0) // page)
        self.held = first + (rng.integers(0, extra + 1, len(self.ctx)) if extra else 0)
        self.pass_held = held
        need = np.maximum(self.held, -(-(np.maximum(self.ctx, 0) + np.maximum(self.new, 0)) // page))
        self.width = int(need.max()) + 2 if width is None else width
        total = int(need.sum()) + spare
        order = rng.permutation(total)
        self.n_pages = total
        self.table = np.full((len(self.ctx), self.width), -1, np.int64)
        u = 0
        for b, h in enumerate(self.held):
            h = min(int(h), self.width)
            self.table[b, :h] = order[u:u + h]
            u += h
        self.free = order[u:]
        self.rows = int(np.maximum(self.new, 0).sum()) + pad
        self.parents = None
        if tree:
            self.parents = np.concatenate([rng.integers(-1, i) if i else -1 for n in self.new for i in range(n)] +
                                          [np.full(pad, -1)], axis=None).astype(np.int64)

    def run(self, **kw):
        dev = {n: i32(getattr(self, n)) for n in ("ctx", "new", "held", "table")}
        free = i32(kw.pop("free", self.free))
        rows = kw.pop("rows", self.rows)
        mask_wanted = kw.pop("mask", True)
        parents = i32(self.parents) if self.parents is not None else None
        B = len(self.ctx)
        out = dict(table=dev["table"], row_start=i32([-7] * (B + 1)), pages=i32([-7] * B), taken=i32([-7]),
                   row_req=i32([-7] * rows), row_pos=i32([-7] * rows), row_slot=i32([-7] * rows),
                   mask=torch.full((rows,), -7, dtype=torch.int64, device=DEV) if mask_wanted else None)
        status = word()
        args = mv.make_map_args(
            n_req=B, n_rows=rows, page_size=self.page, n_pages=kw.pop("n_pages", self.n_pages),
            table_width=self.width, n_free=free.numel(), ctx_len=at(dev["ctx"]), new_len=at(dev["new"]),
            pages_held=at(dev["held"]) if self.pass_held else 0, free_pages=at(free), parents=at(parents),
            block_table=at(out["table"]), row_start=at(out["row_start"]), pages=at(out["pages"]),
            n_taken=at(out["taken"]), row_req=at(out["row_req"]), row_pos=at(out["row_pos"]),
            row_slot=at(out["row_slot"]), tree_mask=at(out["mask"]), dev_status=at(status))
        assert not kw
        mv.moe_round_map(args, stream())
        got = {n: None if t is None else t.cpu().numpy().astype(np.int64) for n, t in out.items()}
        return got, int(status.item())

    def plain(self, free=None, rows=None):
        """Request after request, row after row, for lengths that are consistent."""
        free = self.free if free is None else free
        rows = self.rows if rows is None else rows
        P, table = self.page, self.table.copy()
        row_req, row_pos, row_slot = np.full(rows, -1), np.zeros(rows, np.int64), np.full(rows, -1)
        mask = np.zeros(rows, np.uint64)
        start, pages, f, r = [0], [], 0, 0
        for b in range(len(self.ctx)):
            ctx, new = int(self.ctx[b]), int(self.new[b])
            held = int(self.held[b]) if self.pass_held else -(-ctx // P)
            need = min(-(-(ctx + new) // P), self.width)
            have = held
            for c in range(held, need):
                if f < len(free):
                    table[b, c] = free[f]
                    have += 1
                else:
                    table[b, c] = -1
                f += 1
            pages.append(have)
            masks, depths = [], []
            for i in range(new):
                up = -1 if self.parents is None and i == 0 else i - 1 if self.parents is None else int(self.parents[r])
                m, d = 1 << i if i < 64 else 0, 0
                if up >= 0 and i < 64:
                    m, d = m | masks[up], depths[up] + 1
                elif i >= 64:
                    d = i
                masks.append(m)
                depths.append(d)
                if r < rows:
                    c, o = divmod(ctx + i, P)
                    row_req[r], row_pos[r] = b, ctx + d
                    row_slot[r] = table[b, c] * P + o if c < self.width and table[b, c] >= 0 else -1
                    mask[r] = np.uint64(m)
                r += 1
            start.append(min(r, rows))
        return dict(table=table, row_start=np.array(start), pages=np.array(pages), taken=np.array([min(f, len(free))]),
                    row_req=row_req, row_pos=row_pos, row_slot=row_slot, mask=mask.view(np.int64))


# ---- norm, rotation, cache write -------------------------------------------------------

def rotate64(x, gain, pos, inv_freq, rot, interleaved, eps, scale):
    """[rows][heads][D] in float64, and the largest magnitude of each element's pair before rotation."""
    y = x.double()
    if gain is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * gain.double()
    amp = y.abs()
    if rot:
        angle = pos.double()[:, None, None] * inv_freq
        c, s = torch.cos(angle) * scale, torch.sin(angle) * scale
        i = torch.arange(rot // 2, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[..., ia], y[..., ib]
        y, amp = y.clone(), amp.clone()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        both = torch.maximum(a.abs(), b.abs()) * abs(scale)
        amp[..., ia], amp[..., ib] = both, both
    return y, amp


# ---- attention -------------------------------------------------------------------------

class TreeCase:
    """A ragged batch of trees over a paged cache, filled with NaN wherever no position lives."""

    def __init__(self, seed, ctx, counts, *, hq, hkv, d, page, dtype, layout="nhd", mask="tree", scale=None,
                 q_scale=2.0, max_tree=None, pad_rows=0, q_pad=0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.dt, self.code = DT[dtype]
        self.ctx, self.counts = list(ctx), list(counts)
        self.hq, self.hkv, self.d, self.page = hq, hkv, d, page
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        self.start = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int64)
        self.rows = int(self.start[-1]) + pad_rows
        self.max_tree = max_tree or max(1, max(self.counts))
        need = [-(-(c + n) // page) for c, n in zip(self.ctx, self.counts)]
        self.width = max(max(need), 1) + 1
        self.n_pages = sum(need) + 3
        order, u = rng.permutation(self.n_pages), 0
        self.table = np.full((len(self.ctx), self.width), -1, np.int64)
        shape = (self.n_pages, page, hkv, d) if layout == "nhd" else (self.n_pages, hkv, page, d)
        self.k = torch.full(shape, float("nan"), dtype=self.dt, device=DEV)
        self.v = self.k.clone()
        if layout == "hnd":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        for b, n in enumerate(need):
            self.table[b, :n] = order[u:u + n]
            u += n
            p, o = self.where(b, np.arange(self.ctx[b] + self.counts[b]))
            for cache in (self.k, self.v):
                cache[p, o] = torch.randn((len(p), hkv, d), generator=gen, device=DEV).to(self.dt)
        wide = torch.randn((self.rows, hq * d + q_pad), generator=gen, device=DEV).mul_(q_scale).to(self.dt)
        self.q = wide[:, :hq * d].view(self.rows, hq, d) if q_pad == 0 else wide[:, :hq * d].unflatten(1, (hq, d))
        self.mask = None
        if mask != "chain":
            words = []
            for n in self.counts:
                m = []
                for i in range(n):
                    up = int(rng.integers(-1, i)) if i else -1
                    m.append((1 << i) | (m[up] if up >= 0 else 0))
                if mask == "random":  # any rows at all, now and then none
                    m = [int(rng.integers(0, 1 << 63)) & ((1 << n) - 1) if rng.random() < 0.8 else 0 for _ in range(n)]
                words += m
            words += [0] * pad_rows
            self.mask = torch.from_numpy(np.array(words, np.uint64).view(np.int64)).to(DEV)

    def where(self, b, pos):
        pages = torch.from_numpy(self.table[b][pos // self.page]).to(DEV)
        return pages, torch.from_numpy(pos % self.page).to(DEV)

    def args(self, out, lse, status, table=None, ctx=None, start=None, max_tree=None):
        self.keep = [i32(self.table) if table is None else table, i32(self.ctx) if ctx is None else ctx,
                     i32(self.start) if start is None else start]
        cache = mv.make_kv_cache(at(self.k), at(self.v), n_pages=self.n_pages, page_size=self.page,
                                 page_stride=self.k.stride(0), slot_stride=self.k.stride(1),
                                 head_stride=self.k.stride(2))
        return mv.make_tree_attention_args(
            n_req=len(self.ctx), n_rows=self.rows, max_tree=max_tree or self.max_tree, q_heads=self.hq,
            kv_heads=self.hkv, head_dim=self.d, dtype=self.code, q=at(self.q), q_stride=self.q.stride(0), out=at(out),
            out_stride=out.stride(0), lse=at(lse), row_start=at(self.keep[2]), ctx_len=at(self.keep[1]),
            block_table=at(self.keep[0]), table_width=self.width, tree_mask=at(self.mask), cache=cache,
            scale=self.scale, dev_status=at(status))

    def outputs(self):
        return (torch.full((self.rows, self.hq, self.d), float("nan"), dtype=self.dt, device=DEV),
                torch.full((self.rows, self.hq), float("nan"), device=DEV))

    def run(self, times=1, **kw):
        out, lse = self.outputs()
        status = word()
        args = self.args(out, lse, status, **kw)
        ws = torch.zeros(mv.moe_tree_attention_workspace_bytes(args), dtype=torch.uint8, device=DEV)
        assert ws.numel() > 0
        for _ in range(times):
            mv.moe_tree_attention(args, at(ws), ws.numel(), stream())
        return out, lse, int(status.item())

    def seen(self, b):
        n, ctx = self.counts[b], self.ctx[b]
        seen = torch.zeros((n, ctx + n), dtype=torch.bool, device=DEV)
        seen[:, :ctx] = True
        for i in range(n):
            word_ = (1 << (i + 1)) - 1 if self.mask is None else int(self.mask[self.start[b] + i]) & (2**64 - 1)
            for j in range(n):
                seen[i, ctx + j] = bool((word_ >> j) & 1)
        return seen

    def check(self, out, lse, only=None, weight_step=2**-25):
        """Every request's rows against float64, within the bound that the roundings add up to (weight_step: what an
        fp16 weight below its smallest normal number may be off by, as a share of the largest)."""
        u = torch.finfo(self.dt).eps / 2
        group = self.hq // self.hkv
        for b in range(len(self.ctx)) if only is None else only:
            r0, r1 = int(self.start[b]), int(self.start[b + 1])
            if r1 == r0:
                continue
            total = self.ctx[b] + r1 - r0
            seen = self.seen(b)
            p, o = self.where(b, np.arange(total))
            for h in range(self.hkv):
                k, v = self.k[p, o, h].double(), self.v[p, o, h].double()
                q = self.q[r0:r1, h * group:(h + 1) * group].double()
                s = torch.einsum("ngd,ld->ngl", q, k) * self.scale
                # a 32-bit sum of d products is off by at most (d + 2) roundings of their magnitudes
                ds = (self.d + 2) * 2**-24 * abs(self.scale) * torch.einsum("ngd,ld->ngl", q.abs(), k.abs())
                hide = ~seen[:, None, :]
                s = torch.where(hide, -math.inf, s)
                ds = torch.where(hide, 0, ds).amax(-1)
                none = (~seen.any(-1))[:, None].expand(-1, group)
                ref_lse = torch.logsumexp(s, -1)
                w = torch.exp(s - torch.where(none, 0, ref_lse)[..., None])
                hidden_free = torch.where(seen.any(0)[:, None], v, 0)
                ref, mass = w @ hidden_free, w @ hidden_free.abs()
                # weights rounded to the element type (below its smallest normal number: absolutely)
                tiny = weight_step * hidden_free.abs().sum(0) if self.dt == torch.float16 else 0.0
                bound = u * (ref.abs() + mass * (1 + u)) + mass * (2 * ds[..., None] + 1e-5) + tiny + (
                    2**-24 if self.dt == torch.float16 else 0.0)
                got = out[r0:r1, h * group:(h + 1) * group].double()
                bad = ~((got - ref).abs() <= bound)
                assert not bad.any(), (b, h, int(bad.sum()), float((got - ref).abs().max()))
                assert (got[none] == 0).all()
                g = lse[r0:r1, h * group:(h + 1) * group].double()
                assert ((g == ref_lse) | ((g - ref_lse).abs() <= ds + 4e-6 + 1e-6 * ref_lse.abs())).all(), (b, h)
