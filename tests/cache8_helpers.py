"""Plain implementations in 64 bits of the 8-bit cache's operators, and set-up shared by their tests."""
from __future__ import annotations

import math

import numpy as np
import torch

import spec_verify_layer_gb300 as mv
from round_ops_helpers import DEV, DT, at, i32, stream, word

FORMATS = {"e4m3": (mv.MOE_E4M3, torch.float8_e4m3fn, 448.0), "i8": (mv.MOE_I8, torch.int8, 127.0)}


def code_values(fmt):
    """The value of each of the 256 codes, by the formats' definitions; NaN where a code is."""
    c = np.arange(256)
    if fmt == "i8":
        return np.where(c < 128, c, c - 256).astype(np.float64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0**-9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


def nearest_codes(x, fmt):
    """Codes (0..255) nearest to x (float64, within the largest code), ties to the even one."""
    if fmt == "i8":
        return (np.rint(x).astype(np.int64) & 255).astype(np.uint8)
    values = code_values(fmt)[:127]  # ascending
    mag = np.abs(x)
    hi = np.searchsorted(values, mag).clip(0, 126)
    lo = (hi - 1).clip(0)
    up, down = values[hi] - mag, mag - values[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = np.where(hi == 0, 0, pick)
    return np.where(np.signbit(x), pick | 128, pick).astype(np.uint8)


def least_exponent(most, fmt):
    """The least e >= -126 with most <= largest code * 2^e."""
    top, e = FORMATS[fmt][2], -126
    while most > math.ldexp(top, e):
        e += 1
    return e


class Cache8:
    """A ragged batch's pages, codes and scales."""

    def __init__(self, seed, ctx, counts, *, hkv, d, page, block, fmt, layout="nhd", spare=3, scales="pow2"):
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.ctx, self.counts = list(ctx), list(counts)
        self.hkv, self.d, self.page, self.block, self.fmt = hkv, d, page, block, fmt
        self.code, self.kind, self.top = FORMATS[fmt]
        need = [-(-(c + n) // page) for c, n in zip(self.ctx, self.counts)]
        self.width = max(max(need), 1) + 1
        self.n_pages = sum(need) + spare
        self.start = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int64)
        order, u = self.rng.permutation(self.n_pages), 0
        self.table = np.full((len(self.ctx), self.width), -1, np.int64)
        for b, n in enumerate(need):
            self.table[b, :n] = order[u:u + n]
            u += n
        hnd = layout == "hnd"
        shape = (self.n_pages, hkv, page, d) if hnd else (self.n_pages, page, hkv, d)
        blocks = (self.n_pages, hkv, page // block) if hnd else (self.n_pages, page // block, hkv)
        for name in ("k", "v"):
            x = torch.randn(shape, generator=self.gen, device=DEV).mul_(self.top / 4).clamp_(-self.top, self.top)
            codes = (x.round() if fmt == "i8" else x).to(self.kind)
            e = torch.randint(-1, 2, blocks, generator=self.gen, device=DEV).float()
            if scales != "pow2":
                e = e + torch.rand(blocks, generator=self.gen, device=DEV)
            scale = torch.exp2(e) * 4 / self.top
            if scales == "pow2":
                scale = torch.exp2(torch.log2(scale).round())
            if hnd:
                codes, scale = codes.transpose(1, 2), scale.transpose(1, 2)
            setattr(self, name, codes)
            setattr(self, name + "_scale", scale)

    def where(self, b, pos):
        pages = torch.from_numpy(self.table[b][pos // self.page]).to(DEV)
        return pages, torch.from_numpy(pos % self.page).to(DEV)

    def raw(self, name):
        return getattr(self, name).view(torch.uint8)

    def values(self, name, b, pos):
        """float64 [positions][heads][d]: the 32-bit product of code and scale."""
        p, o = self.where(b, pos)
        codes = torch.from_numpy(code_values(self.fmt)).to(DEV)[self.raw(name)[p, o].long()]
        return (codes.float() * getattr(self, name + "_scale")[p, o // self.block][..., None]).double()

    def cache(self):
        k, s = self.k, self.k_scale
        return mv.make_kv_cache8(at(k), at(self.v), at(s), at(self.v_scale), n_pages=self.n_pages, page_size=self.page,
                                 block_size=self.block, format=self.code, page_stride=k.stride(0), slot_stride=k.stride(1),
                                 head_stride=k.stride(2), scale_page_stride=s.stride(0), scale_block_stride=s.stride(1),
                                 scale_head_stride=s.stride(2))

    def rows_args(self, k, v, status, *, rows=None, table=None, ctx=None, start=None):
        self.keep = [i32(self.start) if start is None else start, i32(self.ctx) if ctx is None else ctx,
                     i32(self.table) if table is None else table]
        code = {t: c for t, c in DT.values()}[k.dtype]
        return mv.make_cache8_args(
            n_req=len(self.ctx), n_rows=k.shape[0] if rows is None else rows, kv_heads=self.hkv, head_dim=self.d, dtype=code,
            k=at(k), v=at(v), k_stride=k.stride(0), v_stride=v.stride(0), row_start=at(self.keep[0]),
            ctx_len=at(self.keep[1]), block_table=at(self.keep[2]), table_width=self.width, cache=self.cache(),
            dev_status=at(status))

    def appended(self, rows, only=None):
        """What an append of `rows` ({"k": [n][heads][d], "v": ...}) makes of codes and scales, block after block."""
        out = {}
        lut = code_values(self.fmt)
        for name in ("k", "v"):
            codes, scale = self.raw(name).cpu().numpy().copy(), getattr(self, name + "_scale").cpu().numpy().copy()
            x = rows[name].double().cpu().numpy()
            for b in range(len(self.ctx)) if only is None else only:
                ctx, n, B = self.ctx[b], self.counts[b], self.block
                for first in range(ctx // B * B, ctx + n if n else 0, B):
                    page, slot = int(self.table[b][first // self.page]), first % self.page
                    if not 0 <= page < self.n_pages:
                        continue
                    held = max(0, min(B, ctx - first))
                    end = min(B, ctx + n - first)
                    for h in range(self.hkv):
                        s = np.float32(scale[page, slot // B, h])
                        s = s if np.isfinite(s) and s >= 2.0**-126 else np.float32(0)
                        old = (lut[codes[page, slot:slot + held, h]].astype(np.float32) * s).astype(np.float64)
                        r = self.start[b] + first - ctx
                        y = np.concatenate([old, x[r + held:r + end, h]])
                        finite = np.abs(np.where(np.isfinite(y), y, 0))
                        e = least_exponent(finite.max(initial=0), self.fmt)
                        y = np.where(np.isnan(y), 0, np.clip(np.ldexp(y, -e), -self.top, self.top))
                        codes[page, slot:slot + end, h] = nearest_codes(y, self.fmt)
                        scale[page, slot // B, h] = np.float32(math.ldexp(1, e))
            out[name], out[name + "_scale"] = codes, scale
        return out

    def same(self, expected):
        for name in ("k", "v"):
            got = self.raw(name).cpu().numpy()
            lut = code_values(self.fmt)
            np.testing.assert_array_equal(lut[got], lut[expected[name]], err_msg=name)  # (+0 and -0 are one value)
            np.testing.assert_array_equal(getattr(self, name + "_scale").cpu().numpy(), expected[name + "_scale"], err_msg=name)


class Tree8Case(Cache8):
    """Trees of drafted rows over an 8-bit cache."""

    def __init__(self, seed, ctx, counts, *, hq, hkv, d, page, block, fmt, dtype="bf16", layout="nhd", mask="tree", scale=None,
                 q_scale=2.0, max_tree=None, pad_rows=0, q_pad=0, scales="any"):
        super().__init__(seed, ctx, counts, hkv=hkv, d=d, page=page, block=block, fmt=fmt, layout=layout, scales=scales)
        self.dt, self.type = DT[dtype]
        self.hq = hq
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        self.rows = int(self.start[-1]) + pad_rows
        self.max_tree = max_tree or max(1, max(self.counts))
        wide = torch.randn((self.rows, hq * d + q_pad), generator=self.gen, device=DEV).mul_(q_scale).to(self.dt)
        self.q = wide[:, :hq * d].unflatten(1, (hq, d))
        self.mask = None
        if mask != "chain":
            words = []
            for n in self.counts:
                m = []
                for i in range(n):
                    up = int(self.rng.integers(-1, i)) if i else -1
                    m.append((1 << i) | (m[up] if up >= 0 else 0))
                if mask == "random":  # any rows at all, now and then none
                    m = [int(self.rng.integers(0, 1 << 63)) & ((1 << n) - 1) if self.rng.random() < 0.8 else 0 for _ in range(n)]
                words += m
            words += [0] * pad_rows
            self.mask = torch.from_numpy(np.array(words, np.uint64).view(np.int64)).to(DEV)

    def args(self, out, lse, status, table=None, ctx=None, start=None, max_tree=None):
        self.keep = [i32(self.table) if table is None else table, i32(self.ctx) if ctx is None else ctx,
                     i32(self.start) if start is None else start]
        return mv.make_tree_attention8_args(
            n_req=len(self.ctx), n_rows=self.rows, max_tree=max_tree or self.max_tree, q_heads=self.hq, kv_heads=self.hkv,
            head_dim=self.d, dtype=self.type, q=at(self.q), q_stride=self.q.stride(0), out=at(out), out_stride=out.stride(0),
            lse=at(lse), row_start=at(self.keep[2]), ctx_len=at(self.keep[1]), block_table=at(self.keep[0]),
            table_width=self.width, tree_mask=at(self.mask), cache=self.cache(), scale=self.scale, dev_status=at(status))

    def outputs(self):
        return (torch.full((self.rows, self.hq, self.d), float("nan"), dtype=self.dt, device=DEV),
                torch.full((self.rows, self.hq), float("nan"), device=DEV))

    def run(self, times=1, **kw):
        out, lse = self.outputs()
        status = word()
        args = self.args(out, lse, status, **kw)
        ws = torch.zeros(mv.moe_tree_attention8_workspace_bytes(args), dtype=torch.uint8, device=DEV)
        assert ws.numel() > 0
        for _ in range(times):
            mv.moe_tree_attention8(args, at(ws), ws.numel(), stream())
        return out, lse, int(status.item())

    def seen(self, b):
        n, ctx = self.counts[b], self.ctx[b]
        seen = torch.zeros((n, ctx + n), dtype=torch.bool, device=DEV)
        seen[:, :ctx] = True
        for i in range(n):
            bits = (1 << (i + 1)) - 1 if self.mask is None else int(self.mask[self.start[b] + i]) & (2**64 - 1)
            for j in range(n):
                seen[i, ctx + j] = bool((bits >> j) & 1)
        return seen

    def check(self, out, lse, only=None, hidden=None, values=None):
        """Every request's rows against float64, within what the roundings add up to:
        scores: a 32-bit sum of d products is off by at most (d + 2) roundings of their magnitudes, and the score as
        a power of two, with the value's scale in it (log2 within 48 of 0), by a few of its own; weights: 2^-11 each,
        below fp16's smallest normal number 2^-32 of the largest weight times scale; the result: half a step."""
        u = torch.finfo(self.dt).eps / 2
        group = self.hq // self.hkv
        for b in range(len(self.ctx)) if only is None else only:
            r0, r1 = int(self.start[b]), int(self.start[b + 1])
            if r1 == r0:
                continue
            total = np.arange(self.ctx[b] + r1 - r0)
            seen = self.seen(b)
            if hidden is not None:
                seen = seen & ~hidden(b)[None]
            k_all, v_all = self.values("k", b, total), self.values("v", b, total)
            if values is not None:
                v_all = values(b, v_all)
            p, o = self.where(b, total)
            vs_all = self.v_scale[p, o // self.block].double()
            for h in range(self.hkv):
                k = torch.where(seen.any(0)[:, None], k_all[:, h], 0.0)
                v = torch.where(seen.any(0)[:, None], v_all[:, h], 0.0)
                q = self.q[r0:r1, h * group:(h + 1) * group].double()
                s = torch.einsum("ngd,ld->ngl", q, k) * self.scale
                ds = (self.d + 2) * 2**-24 * abs(self.scale) * torch.einsum("ngd,ld->ngl", q.abs(), k.abs())
                ds = ds + 2**-22 * (s.abs() + 48)
                hide = ~seen[:, None, :]
                s = torch.where(hide, -math.inf, s)
                ds = torch.where(hide, 0, ds).amax(-1)
                none = (~seen.any(-1))[:, None].expand(-1, group)
                ref_lse = torch.logsumexp(s, -1)
                w = torch.exp(s - torch.where(none, 0, ref_lse)[..., None])
                ref, mass = w @ v, w @ v.abs()
                vs = torch.where(seen.any(0), vs_all[:, h], 0.0)
                codes = torch.where(vs[:, None] > 0, v.abs() / vs.clamp(min=1e-300)[:, None], 0.0)
                tiny = 2**-32 * (w * vs).amax(-1)[..., None] * codes.sum(0)
                bound = u * (ref.abs() + mass) + 2**-11 * mass + mass * 2 * ds[..., None] + tiny + (
                    2**-24 if self.dt == torch.float16 else 0.0)
                got = out[r0:r1, h * group:(h + 1) * group].double()
                wrong = ~((got - ref).abs() <= bound)
                assert not wrong.any(), (b, h, int(wrong.sum()), float((got - ref).abs().max()))
                assert (got[none] == 0).all()
                g = lse[r0:r1, h * group:(h + 1) * group].double()
                assert ((g == ref_lse) | ((g - ref_lse).abs() <= ds + 4e-6 + 1e-6 * ref_lse.abs())).all(), (b, h)
