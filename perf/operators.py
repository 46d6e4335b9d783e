"""Cases of the verify round's attention-side operators, with their plain forms.

A verify round runs, around the expert layers: the page and slot map of the rows to
come (moe_round_map), the per-head norms and rotation of queries and keys with the
write into the paged cache (moe_qk_rope_cache), the attention of a tree of drafted
rows over that cache (moe_tree_attention), and the log probabilities of the drafted
tokens under the logits (moe_token_logprobs).  Where `own` is false, `run` computes an
operator with elementary torch operations in 32 bits (angles in 64); where it is true
it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # six requests of a small server, each with a little tree of drafts: latency
        dict(name="map_verify", op="map", req=6, ctx=4096, new_lo=1, new=16, page=16, tree=True, held=True, pad=7),
        # prompts of many requests admitted at once, chunks appended to what is cached
        dict(name="map_prompts", op="map", req=1500, ctx=20000, new_lo=0, new=1000, page=16, tree=False, held=False,
             pad=0),
        # one token of one request: the plain decode step
        dict(name="rope_token", op="rope", rows=1, hq=32, hkv=4, d=128, rot=128, inter=False, norm=True, page=16,
             pos=5000, layout="nhd", dtype="bf16"),
        # the drafted rows of a full batch; half the head rotated, pairs side by side
        dict(name="rope_batch", op="rope", rows=701, hq=24, hkv=8, d=64, rot=32, inter=True, norm=True, page=32,
             pos=1000000, layout="hnd", dtype="f16"),
        # a prompt chunk
        dict(name="rope_prompt", op="rope", rows=16384, hq=32, hkv=4, d=128, rot=128, inter=False, norm=True, page=64,
             pos=130000, layout="nhd", dtype="bf16"),
        # one row over a short context: the smallest attention call
        dict(name="tree_token", op="tree", req=1, n_lo=1, n=1, ctx_lo=0, ctx=1000, hq=32, hkv=4, d=128, page=16, layout="nhd",
             dtype="bf16", chain=False, spare=1.5),
        # the batch-1 verify round: 16 drafted rows over a long context
        dict(name="tree_verify", op="tree", req=1, n_lo=16, n=16, ctx_lo=0, ctx=32768, hq=32, hkv=4, d=128, page=64,
             layout="nhd", dtype="bf16", chain=False, spare=1.5),
        # a ragged batch: from no row and no context up to 24 rows over 6001 tokens, odd pages
        dict(name="tree_batch", op="tree", req=33, n_lo=0, n=24, ctx_lo=0, ctx=6001, hq=16, hkv=8, d=64, page=24, layout="hnd",
             dtype="f16", chain=False, spare=1.2),
        # full trees over very long contexts in a cache whose offsets pass 32 bits
        dict(name="tree_long", op="tree", req=2, n_lo=40, n=64, ctx_lo=131071, ctx=200001, hq=32, hkv=4, d=128, page=64,
             layout="nhd", dtype="bf16", chain=False, spare=14.0),
        # a few drafted rows, a small odd vocabulary
        dict(name="logp_draft", op="logp", rows=5, vocab=32003, k=5, dtype="f32", masked=False, temp=1.0),
        # a wide verify round: 16 rows, a large vocabulary in 16 bits (many ties)
        dict(name="logp_verify", op="logp", rows=16, vocab=131072, k=20, dtype="bf16", masked=False, temp=0.7),
        # scoring a prompt: many rows, a vocabulary partly masked out
        dict(name="logp_prompt", op="logp", rows=2000, vocab=129283, k=8, dtype="f32", masked=True, temp=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "rope", "tree", "tree", "logp"])
    if op == "map":
        req = _log_int(rng, 1, 2000)
        tree = rng.random() < 0.5
        new = _log_int(rng, 1, 64) if tree else _log_int(rng, 1, max(1, min(4000, 1500000 // req)))
        return dict(op="map", req=req, ctx=_log_int(rng, 1, 60000 if req < 500 else 20000),
                    new_lo=rng.randint(0, min(1, new)), new=new, page=rng.choice([1, 8, 16, 24, 32, 64, 128, 256]),
                    tree=tree, held=rng.random() < 0.5, pad=rng.choice([0, 0, 5, 64]))
    if op == "rope":
        d = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        per_row = (hkv * group + 2 * hkv) * d
        return dict(op="rope", rows=_log_int(rng, 1, max(1, min(16384, 16384 * 40 * 128 // per_row))), hq=hkv * group,
                    hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4]), inter=rng.random() < 0.4,
                    norm=rng.random() < 0.75, page=rng.choice([1, 8, 16, 24, 64, 256]),
                    pos=_log_int(rng, 2, 1000000), layout=rng.choice(["nhd", "hnd"]),
                    dtype=rng.choice(["bf16", "f16"]))
    if op == "tree":
        d = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        req = _log_int(rng, 1, 64)
        n = rng.choice([1, _log_int(rng, 1, 64)])
        # the padded sums of the plain form and the work stay below the largest listed case's
        room = 2 * 200001 * 4 * 128 // (req * hkv * d)
        room = min(room, 2 * 200001 * 64 * 32 // (req * n * hkv * group))
        room = min(room, 2 * 200001 * 64 * 32 * 128 // (req * n * hkv * group * d))
        return dict(op="tree", req=req, n_lo=rng.randint(0, n) if req > 1 else n, n=n,
                    ctx_lo=0, ctx=_log_int(rng, 1, max(2, min(200001, room))), hq=hkv * group, hkv=hkv, d=d,
                    page=rng.choice([1, 8, 16, 24, 32, 64, 128, 256]), layout=rng.choice(["nhd", "hnd"]),
                    dtype=rng.choice(["bf16", "f16"]), chain=rng.random() < 0.25, spare=1.25)
    vocab = _log_int(rng, 1000, 262144)
    return dict(op="logp", rows=_log_int(rng, 1, max(1, min(4096, 2000 * 129283 // vocab))), vocab=vocab,
                k=rng.choice([0, 1, 5, 8, 20, 32]), dtype=rng.choice(["f32", "bf16", "f16"]),
                masked=rng.random() < 0.4, temp=rng.choice([1.0, 0.7, 1.3]))


# ---------------------------------------------------------------- lengths and work

def _lengths(count, lo, hi):
    """`count` lengths spread evenly from lo to hi: their sum goes by the case alone."""
    if count == 1:
        return [hi]
    return [lo + (hi - lo) * i // (count - 1) for i in range(count)]


def _pages(tokens, page):
    return (tokens + page - 1) // page


def work(case):
    c = case
    if c["op"] == "map":
        rows = sum(_lengths(c["req"], c["new_lo"], c["new"])) + c["pad"]
        taken = _pages(sum(_lengths(c["req"], c["new_lo"], c["new"])), c["page"])  # about: by what is held already
        out = rows * (12 + (8 if c["tree"] else 0)) + c["req"] * 8 + 4 * taken
        return {"bytes": out + c["req"] * (12 if c["held"] else 8) + 4 * taken + (4 * rows if c["tree"] else 0),
                "flops": 0}
    if c["op"] == "rope":
        per = (c["hq"] + 2 * c["hkv"]) * c["d"]
        return {"bytes": c["rows"] * (4 * per + 8), "flops": c["rows"] * per * 8}
    if c["op"] == "tree":
        ctx = _lengths(c["req"], c["ctx_lo"], c["ctx"])
        rows = _lengths(c["req"], c["n_lo"], c["n"])
        # which context meets which tree goes by the seed: the mean of it
        kv = sum(ctx) + sum(rows)
        mean_rows = sum(rows) / len(rows)
        size = 2 * sum(rows) * c["hq"] * c["d"] * 2 + sum(rows) * c["hq"] * 4
        return {"bytes": kv * c["hkv"] * c["d"] * 4 + size, "flops": 4 * kv * mean_rows * c["hq"] * c["d"]}
    size = 4 if c["dtype"] == "f32" else 2
    return {"bytes": c["rows"] * (c["vocab"] * size + 16 + 8 * c["k"]), "flops": 4 * c["rows"] * c["vocab"]}


# ---------------------------------------------------------------- inputs

def _shuffled(values, gen):
    return torch.tensor(values, dtype=torch.int32)[torch.randperm(len(values), generator=gen)]


def _parents(lengths, gen):
    """Parents of each request's drafted rows (-1: the context itself), in topological
    order: a row hangs on one of the three rows before it, or starts a branch."""
    n = int(lengths.sum())
    start = torch.repeat_interleave(torch.cumsum(lengths, 0) - lengths, lengths.long())
    i = torch.arange(n) - start
    back = torch.randint(1, 4, (n,), generator=gen)
    return torch.clamp(i - back, min=-1).to(torch.int32)


def _ancestors(parents, start, count, width):
    """[req][width][width] truth values: is row j the row i or an ancestor of it?
    (I + P)^64 of the parent matrix P is positive exactly there."""
    req = count.numel()
    i = torch.arange(width, device=parents.device)
    at = (start[:req, None].long() + i).clamp(max=max(0, parents.numel() - 1))
    p = torch.where(i < count[:, None], parents[at].long(), torch.full_like(at, -1))
    one = ((p[:, :, None] == i) | torch.eye(width, device=parents.device, dtype=torch.bool)).double()
    return torch.linalg.matrix_power(one, 64) > 0


def _mask_bits(anc):
    j = torch.arange(anc.shape[-1], device=anc.device)
    return (anc.long() << j).sum(-1)


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    if c["op"] == "map":
        ctx = _shuffled(_lengths(c["req"], 0, c["ctx"]), host)
        new = _shuffled(_lengths(c["req"], c["new_lo"], c["new"]), host)
        held = (ctx + c["page"] - 1) // c["page"]
        if c["held"]:  # pages kept from drafts that were not accepted
            held = held + torch.randint(0, 3, (c["req"],), generator=host, dtype=torch.int32)
        need = torch.maximum(held, (ctx + new + c["page"] - 1) // c["page"])
        width = _pages(c["ctx"] + c["new"], c["page"]) + 3
        total, owned = int(need.sum()) + 9, int(held.sum())
        order = torch.randperm(total, generator=host).to(torch.int32)
        table = torch.full((c["req"], width), -1, dtype=torch.int32)
        table[torch.arange(width) < held[:, None]] = order[:owned]
        rows = int(new.sum()) + c["pad"]
        s.update(ctx=ctx.to(DEV), new=new.to(DEV), held=held.to(DEV), free=order[owned:].to(DEV), table=table.to(DEV),
                 n_pages=total, rows=rows, row_start=i32(c["req"] + 1), pages=i32(c["req"]), taken=i32(1),
                 row_req=i32(rows), row_pos=i32(rows), row_slot=i32(rows),
                 mask=torch.zeros(rows, dtype=torch.int64, device=DEV) if c["tree"] else None,
                 parents=torch.cat([_parents(new, host), torch.full((c["pad"],), -1, dtype=torch.int32)]).to(DEV)
                 if c["tree"] else None)
    elif c["op"] == "rope":
        dt, rows, d = DTYPES[c["dtype"]], c["rows"], c["d"]
        n_pages = _pages(rows, c["page"]) * 5 // 4 + 1
        qkv = (torch.randn((rows, (c["hq"] + 2 * c["hkv"]), d), generator=gen, device=DEV) * 1.5).to(dt)
        shape = (n_pages, c["page"], c["hkv"], d) if c["layout"] == "nhd" else (n_pages, c["hkv"], c["page"], d)
        k, v = (torch.randn(shape, generator=gen, device=DEV).to(dt) for _ in range(2))
        if c["layout"] == "hnd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        gain = lambda: (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(dt)  # noqa: E731
        s.update(qkv=qkv, q=qkv[:, :c["hq"]], k=qkv[:, c["hq"]:c["hq"] + c["hkv"]], v=qkv[:, c["hq"] + c["hkv"]:],
                 q_out=torch.empty((rows, c["hq"], d), dtype=dt, device=DEV), k_cache=k, v_cache=v,
                 q_gain=gain() if c["norm"] else None, k_gain=gain() if c["norm"] else None,
                 inv_freq=1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"]),
                 pos=torch.randint(0, c["pos"], (rows,), generator=gen, device=DEV, dtype=torch.int32),
                 slot=torch.randperm(n_pages * c["page"], generator=host)[:rows].to(torch.int32).to(DEV))
    elif c["op"] == "tree":
        dt, d = DTYPES[c["dtype"]], c["d"]
        ctx = _shuffled(_lengths(c["req"], c["ctx_lo"], c["ctx"]), host)
        count = _shuffled(_lengths(c["req"], c["n_lo"], c["n"]), host)
        start = torch.cat([torch.zeros(1, dtype=torch.int32), torch.cumsum(count, 0).to(torch.int32)])
        rows = int(start[-1])
        need = (ctx + count + c["page"] - 1) // c["page"]
        width = int(need.max()) + 1
        n_pages = int(int(need.sum()) * c["spare"]) + 1
        table = torch.full((c["req"], width), -1, dtype=torch.int32)
        table[torch.arange(width) < need[:, None]] = torch.randperm(n_pages, generator=host)[:int(need.sum())].to(
            torch.int32)
        shape = (n_pages, c["page"], c["hkv"], d) if c["layout"] == "nhd" else (n_pages, c["hkv"], c["page"], d)
        k, v = (torch.empty(shape, dtype=dt, device=DEV).normal_(generator=gen) for _ in range(2))
        if c["layout"] == "hnd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        parents = torch.full((rows,), -1, dtype=torch.int32)
        if rows:
            parents = _parents(count, host)
        mask = None
        if not c["chain"]:
            at = torch.arange(64) < count[:, None]
            mask = _mask_bits(_ancestors(parents, start, count, 64))[at].to(DEV) if rows else torch.zeros(
                0, dtype=torch.int64, device=DEV)
        s.update(q=(torch.randn((rows, c["hq"], d), generator=gen, device=DEV) * 2.5).to(dt), k_cache=k, v_cache=v,
                 table=table.to(DEV), ctx=ctx.to(DEV), row_start=start.to(DEV), mask=mask, rows=rows,
                 longest=int((ctx + count).max()), scale=1.0 / math.sqrt(d),
                 out=torch.empty((rows, c["hq"], d), dtype=dt, device=DEV),
                 lse=torch.empty((rows, c["hq"]), dtype=torch.float32, device=DEV))
    else:
        dt = DTYPES[c["dtype"]]
        x = torch.randn((c["rows"], c["vocab"]), generator=gen, device=DEV).mul_(2.5)
        peak = torch.randint(0, c["vocab"], (c["rows"], 4), generator=gen, device=DEV)
        x.scatter_add_(1, peak, 4 + 4 * torch.rand((c["rows"], 4), generator=gen, device=DEV))
        if c["masked"]:
            x.masked_fill_(torch.rand((c["rows"], c["vocab"]), generator=gen, device=DEV) < 0.3, -math.inf)
            x[:, 7] = 0.5
        any_token = torch.randint(0, c["vocab"], (c["rows"],), generator=gen, device=DEV)
        token = torch.where(torch.rand(c["rows"], generator=gen, device=DEV) < 0.6, peak[:, 0], any_token)
        f32 = lambda *n: torch.empty(n, dtype=torch.float32, device=DEV)  # noqa: E731
        s.update(logits=x.to(dt), token=token.to(torch.int32), logp=f32(c["rows"]), entropy=f32(c["rows"]),
                 rank=i32(c["rows"]), top_ids=i32(c["rows"], c["k"]), top_logp=f32(c["rows"], c["k"]))
    if own:
        s.update(_plan(s))
    return s


# ---------------------------------------------------------------- the library's calls

def _plan(s):
    """What a program keeps from round to round: the calls' descriptors, the workspace and the status word."""
    import spec_verify_layer_gb300 as mv
    c, status = s["case"], torch.zeros(1, dtype=torch.int32, device=DEV)
    at = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    types = {"bf16": mv.MOE_BF16, "f16": mv.MOE_F16, "f32": mv.MOE_F32}
    ws = None
    if c["op"] in ("rope", "tree"):
        k = s["k_cache"]
        cache = mv.make_kv_cache(at(k), at(s["v_cache"]), n_pages=k.shape[0], page_size=c["page"],
                                 page_stride=k.stride(0), slot_stride=k.stride(1), head_stride=k.stride(2))
    if c["op"] == "map":
        args = mv.make_map_args(
            n_req=c["req"], n_rows=s["rows"], page_size=c["page"], n_pages=s["n_pages"], table_width=s["table"].shape[1],
            n_free=s["free"].numel(), ctx_len=at(s["ctx"]), new_len=at(s["new"]),
            pages_held=at(s["held"]) if c["held"] else 0, free_pages=at(s["free"]), parents=at(s["parents"]),
            block_table=at(s["table"]), row_start=at(s["row_start"]), pages=at(s["pages"]), n_taken=at(s["taken"]),
            row_req=at(s["row_req"]), row_pos=at(s["row_pos"]), row_slot=at(s["row_slot"]), tree_mask=at(s["mask"]),
            dev_status=at(status))
    elif c["op"] == "rope":
        args = mv.make_qk_rope_args(
            n_rows=c["rows"], q_heads=c["hq"], kv_heads=c["hkv"], head_dim=c["d"], rot_dim=c["rot"],
            interleaved=c["inter"], dtype=types[c["dtype"]], q=at(s["q"]), k=at(s["k"]), v=at(s["v"]),
            q_stride=s["q"].stride(0), k_stride=s["k"].stride(0), v_stride=s["v"].stride(0), q_out=at(s["q_out"]),
            q_out_stride=s["q_out"].stride(0), q_gain=at(s["q_gain"]), k_gain=at(s["k_gain"]),
            inv_freq=at(s["inv_freq"]), row_pos=at(s["pos"]), row_slot=at(s["slot"]), cache=cache, eps=1e-6,
            rot_scale=1.0, dev_status=at(status))
    elif c["op"] == "tree":
        args = mv.make_tree_attention_args(
            n_req=c["req"], n_rows=s["rows"], max_tree=c["n"], q_heads=c["hq"], kv_heads=c["hkv"], head_dim=c["d"],
            dtype=types[c["dtype"]], q=at(s["q"]), q_stride=s["q"].stride(0), out=at(s["out"]),
            out_stride=s["out"].stride(0), lse=at(s["lse"]), row_start=at(s["row_start"]), ctx_len=at(s["ctx"]),
            block_table=at(s["table"]), table_width=s["table"].shape[1], tree_mask=at(s["mask"]), cache=cache,
            scale=s["scale"], dev_status=at(status))
        ws = torch.zeros(mv.moe_tree_attention_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    else:
        args = mv.make_logprob_args(
            n_rows=c["rows"], vocab=c["vocab"], top_k=c["k"], dtype=types[c["dtype"]], logits=at(s["logits"]),
            stride=s["logits"].stride(0), tokens=at(s["token"]), inv_temperature=1.0 / c["temp"], logp=at(s["logp"]),
            entropy=at(s["entropy"]), rank=at(s["rank"]), top_ids=at(s["top_ids"]) if c["k"] else 0,
            top_logp=at(s["top_logp"]) if c["k"] else 0, dev_status=at(status))
        ws = torch.zeros(mv.moe_token_logprobs_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    return {"mv": mv, "args": args, "status": status, "ws": ws}


def _run_own(s):
    mv, op, stream = s["mv"], s["case"]["op"], torch.cuda.current_stream().cuda_stream
    if op == "map":
        mv.moe_round_map(s["args"], stream)
        return _map_outputs(s, *(s[n] for n in ("table", "row_start", "pages", "taken", "row_req", "row_pos",
                                                "row_slot", "mask")))
    if op == "rope":
        mv.moe_qk_rope_cache(s["args"], stream)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "tree":
        mv.moe_tree_attention(s["args"], s["ws"].data_ptr(), s["ws"].numel(), stream)
        return {"out": s["out"], "lse": s["lse"]}
    mv.moe_token_logprobs(s["args"], s["ws"].data_ptr(), s["ws"].numel(), stream)
    return {n: s[n] for n in ("logp", "entropy", "rank", "top_ids", "top_logp")}


# ---------------------------------------------------------------- the plain forms

def _map_outputs(s, table, row_start, pages, taken, row_req, row_pos, row_slot, mask):
    out = {"table": table, "row_start": row_start, "pages": pages, "taken": taken, "row_req": row_req,
           "row_pos": row_pos, "row_slot": row_slot}
    if mask is not None:
        out["mask"] = mask
    return out


def _plain_map(s):
    c, ctx, new, page = s["case"], s["ctx"].long(), s["new"].long(), s["case"]["page"]
    first = (ctx + page - 1) // page
    held = s["held"].long() if c["held"] else first
    pages = torch.maximum(held, (ctx + new + page - 1) // page)
    take = pages - held
    at = torch.cumsum(take, 0) - take
    col = torch.arange(s["table"].shape[1], device=DEV)
    fresh = (col >= held[:, None]) & (col < pages[:, None])
    pick = (at[:, None] + col - held[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][pick], s["table"])
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    row = torch.arange(s["rows"], device=DEV)
    req = torch.searchsorted(start[1:], row, right=True)
    live = req < c["req"]
    req = req.clamp(max=c["req"] - 1)
    i = row - start[req]
    where = ctx[req] + i
    slot = table[req, torch.where(live, where // page, 0)].long() * page + where % page
    depth, mask = i, None
    if c["tree"]:
        anc = _ancestors(s["parents"], start, new, 64)
        i = i.clamp(0, 63)
        depth = anc.sum(-1)[req, i] - 1
        mask = torch.where(live, _mask_bits(anc)[req, i], 0)
    return _map_outputs(s, table, start.int(), pages.int(), take.sum().int()[None],
                        torch.where(live, req, -1).int(), torch.where(live, ctx[req] + depth, 0).int(),
                        torch.where(live, slot, -1).int(), mask)


def _plain_rotate(s, x, gain):
    c, half = s["case"], s["case"]["rot"] // 2
    y = x.float()
    if gain is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * gain.float()
    angle = s["pos"].double()[:, None, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    r = y[..., :c["rot"]]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if c["inter"] else torch.cat([a, b], -1)
    return torch.cat([r, y[..., c["rot"]:]], -1).to(x.dtype)


def _plain_rope(s):
    slot, page = s["slot"].long(), s["case"]["page"]
    s["k_cache"][slot // page, slot % page] = _plain_rotate(s, s["k"], s["k_gain"])
    s["v_cache"][slot // page, slot % page] = s["v"]
    return {"q": _plain_rotate(s, s["q"], s["q_gain"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_tree(s):
    c, rows, req = s["case"], s["rows"], s["case"]["req"]
    hkv, group, d, width, page = c["hkv"], c["hq"] // c["hkv"], c["d"], c["n"], c["page"]
    start = s["row_start"].long()
    count = start[1:] - start[:-1]
    ctx = s["ctx"].long()
    # keys and values of every request, padded to the longest
    col = torch.arange(s["longest"], device=DEV)
    live = col < (ctx + count)[:, None]
    page_of = s["table"].long()[:, col // page].clamp(min=0)
    k = s["k_cache"][page_of, (col % page).expand(req, -1)].float()
    v = s["v_cache"][page_of, (col % page).expand(req, -1)].float() * live[:, :, None, None]
    # the rows, padded to the widest tree
    i = torch.arange(width, device=DEV)
    at = (start[:-1, None] + i).clamp(max=max(0, rows - 1))
    q = s["q"].float()[at].view(req, width, hkv, group, d)
    score = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(req, hkv, group * width, d), k.permute(0, 2, 3, 1))
    node = col - ctx[:, None]
    if s["mask"] is None:
        seen = node[:, None, :] <= i[:, None]
    else:
        bit = (s["mask"][at][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1
        seen = (node < 0)[:, None, :] | (bit == 1)
    seen = (seen & live[:, None, :])[:, None, None]
    score = score.view(req, hkv, group, width, -1).mul_(s["scale"]).masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp_(score.sub_(torch.where(top == -math.inf, 0, top)))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(req, hkv, group * width, -1), v.permute(0, 2, 1, 3)).view(req, hkv, group, width, d)
    out = (out / torch.where(total > 0, total, 1)).permute(0, 3, 1, 2, 4).reshape(req, width, c["hq"], d)
    lse = (top + torch.log(total)).permute(0, 3, 1, 2, 4).reshape(req, width, c["hq"])
    # back from the padded rows
    row = torch.arange(rows, device=DEV)
    of = torch.searchsorted(start[1:], row, right=True)
    return {"out": out[of, row - start[of]].to(s["q"].dtype), "lse": lse[of, row - start[of]]}


def _plain_logp(s):
    c, x, vocab = s["case"], s["logits"].float(), s["case"]["vocab"]
    z = x * (1.0 / c["temp"])
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total[:, 0] - torch.where(e > 0, e * (z - top), 0).sum(-1) / total[:, 0]
    t = s["token"].long()[:, None]
    xt, col = x.gather(1, t), torch.arange(vocab, device=DEV)
    rank = ((x > xt) | ((x == xt) & (col < t))).sum(-1)
    logp = (z.gather(1, t) - top - log_total)[:, 0]
    # whole numbers in the order of (logit, then the lower id)
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 32) + (vocab - 1 - col)
    ids = vocab - 1 - (torch.topk(key, c["k"], -1).values & 0xFFFFFFFF)
    found = z.gather(1, ids)
    none = found == -math.inf
    return {"logp": logp, "entropy": entropy, "rank": rank.int(), "top_ids": torch.where(none, -1, ids).int(),
            "top_logp": torch.where(none, -math.inf, found - top - log_total)}


def run(state):
    if own:
        return _run_own(state)
    return {"map": _plain_map, "rope": _plain_rope, "tree": _plain_tree, "logp": _plain_logp}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rope(s):
    c = s["case"]
    theta = s["pos"].double()[:, None] * s["inv_freq"][None]
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]

    def rotated(x, gain):
        y = x.double()
        if gain is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["d"] + 1e-6) * gain.double()
        pair = y[..., :c["rot"]]
        pair = pair.unflatten(-1, (-1, 2)) if c["inter"] else pair.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if c["inter"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), y[..., c["rot"]:]], -1)

    k, v = s["k_cache"].double(), s["v_cache"].double()
    page, off = s["slot"].long() // c["page"], s["slot"].long() % c["page"]
    k[page, off] = rotated(s["k"], s["k_gain"])
    v[page, off] = s["v"].double()
    return {"q": rotated(s["q"], s["q_gain"]), "k_cache": k, "v_cache": v}


def _exact_tree(s):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    start, ctx = s["row_start"].tolist(), s["ctx"].tolist()
    for b in range(c["req"]):
        r0, r1 = start[b], start[b + 1]
        n, length = r1 - r0, ctx[b] + r1 - r0
        if n == 0:
            continue
        seen = torch.ones((n, length), dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            seen[:, ctx[b]:] = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
        else:
            words = s["mask"][r0:r1].tolist()
            seen[:, ctx[b]:] = torch.tensor([[(w >> j) & 1 == 1 for j in range(n)] for w in words], device=DEV)
        position = torch.arange(length, device=DEV)
        pages = s["table"][b].long()[position // c["page"]]
        for h in range(c["hkv"]):
            k = s["k_cache"][pages, position % c["page"], h].double()
            v = s["v_cache"][pages, position % c["page"], h].double()
            for g in range(h * group, (h + 1) * group):
                x = (s["q"][r0:r1, g].double() @ k.T * s["scale"]).masked_fill(~seen, -math.inf)
                lse[r0:r1, g] = torch.logsumexp(x, -1)
                out[r0:r1, g] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


def _exact_logp(s):
    c = s["case"]
    z = s["logits"].double() * float(np.float32(1.0 / c["temp"]))
    lse = torch.logsumexp(z, -1, keepdim=True)
    top = torch.topk(z, c["k"], -1, sorted=True).values - lse
    logp = (z.gather(1, s["token"].long()[:, None]) - lse)[:, 0]
    z -= lse
    entropy = -(torch.exp(z) * torch.nan_to_num(z, neginf=0.0)).sum(-1)
    return {"logp": logp, "entropy": entropy, "rank": None, "top_ids": None, "top_logp": top}


def exact(case, seed):
    if case["op"] == "map":
        return None  # whole numbers: compared as they are
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "logp": _exact_logp}[case["op"]](s)
