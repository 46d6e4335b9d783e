"""Cases of the 8-bit cache of a verify round and of the check of its drafted tokens, with their plain forms.

The cache of keys and values may be held in 8 bits, codes with a scale for each block of
tokens and head: rows are quantised as they are appended (moe_cache8_append), read back
for whatever wants 16 bits (moe_cache8_read), and attended to by the drafted rows
(moe_tree_attention8).  At the round's end the drafted tokens are accepted or rejected
against the target's probabilities, from given random numbers (moe_verify_drafts).  Where
`own` is false, `run` computes an operator with elementary torch operations in 32 bits
(sums and comparisons of the verification in 64: a draft stands or falls by them); where
it is true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
# codes: their torch type, the largest, as fraction and exponent (largest = fraction * 2^exponent)
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0, 0.875, 9), "i8": (torch.int8, 127.0, 0.9921875, 7)}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of one request joins its block: latency
        dict(name="append_token", op="append", req=1, n_lo=1, n=1, ctx=5000, hkv=4, d=128, page=16, block=16,
             layout="nhd", dtype="bf16", fmt="e4m3"),
        # the drafted rows of a full batch, blocks begun before and behind; odd pages
        dict(name="append_round", op="append", req=200, n_lo=0, n=9, ctx=9000, hkv=8, d=64, page=24, block=8,
             layout="hnd", dtype="f16", fmt="i8"),
        # long prompts written at once
        dict(name="append_prompt", op="append", req=3, n_lo=20011, n=32768, ctx=131, hkv=4, d=128, page=64, block=16,
             layout="nhd", dtype="bf16", fmt="e4m3"),
        # a shared prefix handed to a prompt's attention in 16 bits
        dict(name="read_prefix", op="read", req=1, n_lo=1500, n=1500, ctx=0, hkv=4, d=128, page=16, block=16,
             layout="nhd", dtype="bf16", fmt="e4m3"),
        # long contexts moved out of the cache
        dict(name="read_long", op="read", req=5, n_lo=1001, n=65536, ctx=77, hkv=8, d=64, page=64, block=32,
             layout="hnd", dtype="f16", fmt="i8"),
        # one row over a short context: the smallest attention call
        dict(name="attn8_token", op="attn", req=1, n_lo=1, n=1, ctx_lo=0, ctx=1000, hq=32, hkv=4, d=128, page=16,
             block=16, layout="nhd", dtype="bf16", fmt="e4m3", chain=False, spare=1.5, pow2=True),
        # the decode step of a batch of requests
        dict(name="attn8_decode", op="attn", req=64, n_lo=1, n=1, ctx_lo=4096, ctx=8192, hq=32, hkv=4, d=128, page=64,
             block=64, layout="nhd", dtype="bf16", fmt="e4m3", chain=True, spare=1.1, pow2=True),
        # a ragged batch: from no row and no context up to 24 rows over 6001 tokens, odd pages, scales of any value
        dict(name="attn8_batch", op="attn", req=33, n_lo=0, n=24, ctx_lo=0, ctx=6001, hq=16, hkv=8, d=64, page=24,
             block=8, layout="hnd", dtype="f16", fmt="i8", chain=False, spare=1.2, pow2=False),
        # full trees over very long contexts in a cache whose offsets pass 32 bits
        dict(name="attn8_long", op="attn", req=2, n_lo=40, n=64, ctx_lo=131071, ctx=200001, hq=32, hkv=4, d=128,
             page=64, block=32, layout="nhd", dtype="bf16", fmt="e4m3", chain=False, spare=27.0, pow2=True),
        # the drafts of one request, found by lookup: a small odd vocabulary
        dict(name="verify_one", op="verify", req=1, n_lo=5, n=5, vocab=32003, dtype="f32", mode="lookup", tree=False,
             masked=False, temp=1.0),
        # a batch of drafted chains with the probabilities that they were drawn from
        dict(name="verify_batch", op="verify", req=64, n_lo=1, n=8, vocab=131072, dtype="bf16", mode="drawn",
             tree=False, masked=False, temp=0.8),
        # trees of likely tokens over a large vocabulary partly masked out
        dict(name="verify_trees", op="verify", req=24, n_lo=8, n=48, vocab=129283, dtype="f32", mode="lookup",
             tree=True, masked=True, temp=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


PAGES = [(1, 1), (16, 16), (16, 4), (24, 8), (32, 32), (64, 16), (64, 1), (128, 128), (256, 64)]  # and blocks


def draw(rng):
    op = rng.choice(["append", "append", "read", "attn", "attn", "attn", "verify", "verify"])
    page, block = rng.choice(PAGES)
    common = dict(page=page, block=block, layout=rng.choice(["nhd", "hnd"]), fmt=rng.choice(["e4m3", "i8"]))
    if op in ("append", "read"):
        d, hkv, req = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8]), _log_int(rng, 1, 600)
        n = _log_int(rng, 1, max(1, min(32768, 3 * 26000 * 4 * 128 // (req * hkv * d))))
        return dict(op=op, req=req, n_lo=rng.randint(0, n) if req > 1 else n, n=n, ctx=_log_int(rng, 1, 9000), hkv=hkv,
                    d=d, dtype=rng.choice(["bf16", "f16", "f32"]), **common)
    if op == "attn":
        d, hkv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        req = _log_int(rng, 1, 64)
        n = rng.choice([1, _log_int(rng, 1, 64)])
        # the padded sums of the plain form and the work stay below the largest listed case's
        room = 2 * 200001 * 4 * 128 // (req * hkv * d)
        room = min(room, 2 * 200001 * 64 * 32 // (req * n * hkv * group))
        room = min(room, 2 * 200001 * 64 * 32 * 128 // (req * n * hkv * group * d))
        return dict(op="attn", req=req, n_lo=rng.randint(0, n) if req > 1 else n, n=n, ctx_lo=0,
                    ctx=_log_int(rng, 1, max(2, min(200001, room))), hq=hkv * group, hkv=hkv, d=d,
                    dtype=rng.choice(["bf16", "f16"]), chain=rng.random() < 0.25, spare=1.25, pow2=rng.random() < 0.6,
                    **common)
    vocab = _log_int(rng, 1000, 262144)
    req = _log_int(rng, 1, max(1, min(300, 24 * 28 * 129283 // vocab)))
    n = _log_int(rng, 1, max(1, min(64, 24 * 48 * 129283 // (vocab * req))))
    mode = rng.choice(["greedy", "lookup", "drawn"])
    return dict(op="verify", req=req, n_lo=rng.randint(0, n) if req > 1 else n, n=n, vocab=vocab,
                dtype=rng.choice(["f32", "bf16", "f16"]), mode=mode, tree=mode != "drawn" and rng.random() < 0.6,
                masked=rng.random() < 0.4, temp=rng.choice([1.0, 0.7, 1.3]))


# ---------------------------------------------------------------- lengths and work

def _lengths(count, lo, hi):
    """`count` lengths spread evenly from lo to hi: their sum goes by the case alone."""
    if count == 1:
        return [hi]
    return [lo + (hi - lo) * i // (count - 1) for i in range(count)]


def work(case):
    c = case
    rows = sum(_lengths(c["req"], c["n_lo"], c["n"]))
    if c["op"] in ("append", "read"):
        per = 2 * c["hkv"] * c["d"]
        return {"bytes": rows * per * (SIZES[c["dtype"]] + 1) + 8 * c["hkv"] * -(-rows // c["block"]),
                "flops": 2 * rows * per}
    if c["op"] == "attn":
        # which context meets which tree goes by the seed: the mean of it
        kv = sum(_lengths(c["req"], c["ctx_lo"], c["ctx"])) + rows
        size = 4 * rows * c["hq"] * c["d"] + 4 * rows * c["hq"] + 8 * c["hkv"] * -(-kv // c["block"])
        return {"bytes": 2 * kv * c["hkv"] * c["d"] + size, "flops": 4 * kv * (rows / c["req"]) * c["hq"] * c["d"]}
    # logits of the rows that drafts hang on, and for the last token a row of noise and of draft probabilities
    size = SIZES[c["dtype"]]
    inner = max(1, rows // 2 if c["tree"] else rows - c["req"])
    last = {"greedy": 0, "lookup": 4, "drawn": 4 + size}[c["mode"]]
    return {"bytes": c["vocab"] * ((rows if c["mode"] == "greedy" else inner) * size + c["req"] * last) + 24 * rows,
            "flops": 4 * c["vocab"] * inner}


# ---------------------------------------------------------------- inputs

def _shuffled(values, gen):
    return torch.tensor(values, dtype=torch.int32)[torch.randperm(len(values), generator=gen)]


def _parents(lengths, gen, roots):
    """Parents of each request's rows, in topological order: a row hangs on one of the three rows before
    it, or, with roots, starts a branch (-1); without, the first row is the root."""
    n = int(lengths.sum())
    start = torch.repeat_interleave(torch.cumsum(lengths, 0) - lengths, lengths.long())
    i = torch.arange(n) - start
    back = torch.randint(1, 4, (n,), generator=gen)
    up = torch.clamp(i - back, min=-1 if roots else 0)
    return torch.where(i == 0, -1, up).to(torch.int32)


def _ancestors(parents, start, count, width):
    """[req][width][width] truth values: is row j the row i or an ancestor of it?
    (I + P)^64 of the parent matrix P is positive exactly there."""
    i = torch.arange(width, device=parents.device)
    at = (start[:count.numel(), None].long() + i).clamp(max=max(0, parents.numel() - 1))
    p = torch.where(i < count[:, None], parents[at].long(), torch.full_like(at, -1))
    one = ((p[:, :, None] == i) | torch.eye(width, device=parents.device, dtype=torch.bool)).double()
    return torch.linalg.matrix_power(one, 64) > 0


def _codes(shape, fmt, gen):
    """Codes as a calibrated block holds them: a bell whose far end is near the largest code."""
    kind, top, _, _ = FORMATS[fmt]
    out = torch.empty(shape, dtype=kind, device=DEV)
    step = max(1, (1 << 28) // max(1, out[0].numel()))
    for at in range(0, shape[0], step):
        part = out[at:at + step]
        x = torch.empty(part.shape, dtype=torch.float16, device=DEV).normal_(generator=gen).mul_(top / 4)
        part.copy_(x.clamp_(-top, top).round_() if fmt == "i8" else x.clamp_(-top, top))
    return out


def _prepare_cache(c, host, gen, s):
    """Lengths, pages and a cache that is full of codes."""
    count = _shuffled(_lengths(c["req"], c["n_lo"], c["n"]), host)
    ctx = _shuffled(_lengths(c["req"], c.get("ctx_lo", 0), c["ctx"]), host)
    start = torch.cat([torch.zeros(1, dtype=torch.int32), torch.cumsum(count, 0).to(torch.int32)])
    need = (ctx + count + c["page"] - 1) // c["page"]
    total, width = int(need.sum()), int(need.max()) + 1
    # (which context meets which rows goes by the seed, the cache's size does not)
    most = int(((ctx + c["page"] - 1) // c["page"] + (count + c["page"] - 1) // c["page"]).sum())
    n_pages = int(most * c.get("spare", 1.1)) + 1
    table = torch.full((c["req"], width), -1, dtype=torch.int32)
    table[torch.arange(width) < need[:, None]] = torch.randperm(n_pages, generator=host)[:total].to(torch.int32)
    shape, blocks = (n_pages, c["page"], c["hkv"], c["d"]), (n_pages, c["page"] // c["block"], c["hkv"])
    if c["layout"] == "hnd":
        shape, blocks = (n_pages, c["hkv"], c["page"], c["d"]), (n_pages, c["hkv"], c["page"] // c["block"])
    s.update(ctx=ctx.to(DEV), count=count.to(DEV), row_start=start.to(DEV), table=table.to(DEV), rows=int(start[-1]),
             longest=int((ctx + count).max()))
    for name in ("k", "v"):
        codes = _codes(shape, c["fmt"], gen)
        # values of about one: a block's scale is some power of two, or anything near where a program calibrated it
        size = torch.randint(-1, 2, blocks, generator=gen, device=DEV).float()
        if not c.get("pow2", True):
            size = size + torch.rand(blocks, generator=gen, device=DEV)
        scale = torch.exp2(size) * (2.0 ** -7 if c["fmt"] == "e4m3" else 2.0 ** -5)
        if c["layout"] == "hnd":
            codes, scale = codes.transpose(1, 2), scale.transpose(1, 2)
        s.update({name + "_cache": codes, name + "_scale": scale})


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "verify":
        _prepare_verify(c, host, gen, s)
    else:
        _prepare_cache(c, host, gen, s)
        dt, rows = DTYPES[c["dtype"]], s["rows"]
        if c["op"] == "append":
            # keys and values as they come out of one projection; now and then a row of large ones
            kv = torch.randn((rows, 2 * c["hkv"], c["d"]), generator=gen, device=DEV)
            kv *= torch.exp2(torch.randn((rows, 2 * c["hkv"], 1), generator=gen, device=DEV))
            kv = kv.to(dt)
            s.update(k=kv[:, :c["hkv"]], v=kv[:, c["hkv"]:])
        elif c["op"] == "read":
            s.update(k=torch.empty((rows, c["hkv"], c["d"]), dtype=dt, device=DEV),
                     v=torch.empty((rows, c["hkv"], c["d"]), dtype=dt, device=DEV))
        else:
            mask = None
            if not c["chain"]:
                mask = torch.zeros(0, dtype=torch.int64, device=DEV)
                if rows:
                    count = s["count"].cpu()
                    anc = _ancestors(_parents(count, host, True), s["row_start"].cpu(), count, 64)
                    word = (anc.long() << torch.arange(64)).sum(-1)
                    mask = word[torch.arange(64) < count[:, None]].to(DEV)
            s.update(q=(torch.randn((rows, c["hq"], c["d"]), generator=gen, device=DEV) * 2).to(dt), mask=mask,
                     scale=1.0 / math.sqrt(c["d"]), out=torch.empty((rows, c["hq"], c["d"]), dtype=dt, device=DEV),
                     lse=torch.empty((rows, c["hq"]), dtype=torch.float32, device=DEV))
    if own:
        s.update(_plan(s))
    return s


def _prepare_verify(c, host, gen, s):
    count = _shuffled(_lengths(c["req"], c["n_lo"], c["n"]), host)
    start = torch.cat([torch.zeros(1, dtype=torch.int32), torch.cumsum(count, 0).to(torch.int32)])
    rows, vocab, dt = int(start[-1]), c["vocab"], DTYPES[c["dtype"]]
    parents = _parents(count, host, False) if c["tree"] else torch.where(
        torch.arange(rows) == start[:-1].repeat_interleave(count.long()), -1,
        torch.arange(rows) - start[:-1].repeat_interleave(count.long()) - 1).to(torch.int32)
    first = start[:-1].repeat_interleave(count.long())
    above = (first + parents.clamp(min=0)).long().to(DEV)  # the row whose logits a row's token is tested against
    x = torch.randn((rows, vocab), generator=gen, device=DEV).mul_(2.0)
    peak = torch.randint(0, vocab, (rows, 6), generator=gen, device=DEV)
    x.scatter_add_(1, peak, 7 + 4 * torch.rand((rows, 6), generator=gen, device=DEV))
    if c["masked"]:
        x.masked_fill_(torch.rand((rows, vocab), generator=gen, device=DEV) < 0.3, -math.inf)
    x = x.to(dt)
    drawn = None
    if c["mode"] == "drawn":
        # a drafter that knows the target's logits roughly: its probabilities, and a token drawn from them
        q = x[above].float() + torch.randn((rows, vocab), generator=gen, device=DEV)
        q = torch.softmax(q / c["temp"], -1).to(dt)
        race = torch.empty((rows, vocab), device=DEV).exponential_(generator=gen)
        token, drawn = (q.float() / race).argmax(-1), q
    else:
        # one of the likely tokens, sometimes anything, sometimes none
        token = peak[above, torch.randint(0, 6, (rows,), generator=gen, device=DEV)]
        odd = torch.rand(rows, generator=gen, device=DEV)
        token = torch.where(odd < 0.1, torch.randint(0, vocab, (rows,), generator=gen, device=DEV), token)
        token = torch.where(odd > 0.97, -1, token)
    s.update(row_start=start.to(DEV), count=count.to(DEV), rows=rows, parents=parents.to(DEV) if c["tree"] else None,
             logits=x, tokens=token.to(torch.int32), draft_probs=drawn,
             uniform=torch.rand(rows, generator=gen, device=DEV),
             noise=None if c["mode"] == "greedy" else torch.empty((c["req"], vocab), device=DEV).exponential_(
                 generator=gen),
             accepted=torch.zeros(c["req"], dtype=torch.int32, device=DEV),
             path=torch.zeros(rows, dtype=torch.int32, device=DEV),
             next_token=torch.zeros(c["req"], dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------- the library's calls

def _plan(s):
    """What a program keeps from round to round: the calls' descriptors, the workspace and the status word."""
    import spec_verify_layer_gb300 as mv
    c, status = s["case"], torch.zeros(1, dtype=torch.int32, device=DEV)
    at = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    types = {"bf16": mv.MOE_BF16, "f16": mv.MOE_F16, "f32": mv.MOE_F32}
    ws = None
    if c["op"] != "verify":
        k, scale = s["k_cache"], s["k_scale"]
        cache = mv.make_kv_cache8(
            at(k), at(s["v_cache"]), at(scale), at(s["v_scale"]), n_pages=k.shape[0], page_size=c["page"],
            block_size=c["block"], format={"e4m3": mv.MOE_E4M3, "i8": mv.MOE_I8}[c["fmt"]], page_stride=k.stride(0),
            slot_stride=k.stride(1), head_stride=k.stride(2), scale_page_stride=scale.stride(0),
            scale_block_stride=scale.stride(1), scale_head_stride=scale.stride(2))
    if c["op"] in ("append", "read"):
        args = mv.make_cache8_args(
            n_req=c["req"], n_rows=s["rows"], kv_heads=c["hkv"], head_dim=c["d"], dtype=types[c["dtype"]], k=at(s["k"]),
            v=at(s["v"]), k_stride=s["k"].stride(0), v_stride=s["v"].stride(0), row_start=at(s["row_start"]),
            ctx_len=at(s["ctx"]), block_table=at(s["table"]), table_width=s["table"].shape[1], cache=cache,
            dev_status=at(status))
    elif c["op"] == "attn":
        args = mv.make_tree_attention8_args(
            n_req=c["req"], n_rows=s["rows"], max_tree=c["n"], q_heads=c["hq"], kv_heads=c["hkv"], head_dim=c["d"],
            dtype=types[c["dtype"]], q=at(s["q"]), q_stride=s["q"].stride(0), out=at(s["out"]),
            out_stride=s["out"].stride(0), lse=at(s["lse"]), row_start=at(s["row_start"]), ctx_len=at(s["ctx"]),
            block_table=at(s["table"]), table_width=s["table"].shape[1], tree_mask=at(s["mask"]), cache=cache,
            scale=s["scale"], dev_status=at(status))
        ws = torch.zeros(mv.moe_tree_attention8_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    else:
        args = mv.make_verify_args(
            n_req=c["req"], n_rows=s["rows"], vocab=c["vocab"], dtype=types[c["dtype"]], logits=at(s["logits"]),
            stride=s["logits"].stride(0), row_start=at(s["row_start"]), parents=at(s["parents"]), tokens=at(s["tokens"]),
            draft_probs=at(s["draft_probs"]), draft_dtype=types[c["dtype"]], draft_stride=c["vocab"],
            uniform=at(s["uniform"]), noise=at(s["noise"]), noise_stride=c["vocab"],
            inv_temperature=math.inf if c["mode"] == "greedy" else 1.0 / c["temp"], accepted=at(s["accepted"]),
            path=at(s["path"]), next_token=at(s["next_token"]), dev_status=at(status))
        ws = torch.zeros(mv.moe_verify_drafts_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    return {"mv": mv, "args": args, "status": status, "ws": ws}


def _run_own(s):
    mv, op, stream = s["mv"], s["case"]["op"], torch.cuda.current_stream().cuda_stream
    if op == "append":
        mv.moe_cache8_append(s["args"], stream)
        return _cache_state(s)
    if op == "read":
        mv.moe_cache8_read(s["args"], stream)
        return {"k": s["k"], "v": s["v"]}
    if op == "attn":
        mv.moe_tree_attention8(s["args"], s["ws"].data_ptr(), s["ws"].numel(), stream)
        return {"out": s["out"], "lse": s["lse"]}
    mv.moe_verify_drafts(s["args"], s["ws"].data_ptr(), s["ws"].numel(), stream)
    return {n: s[n] for n in ("accepted", "path", "next_token")}


# ---------------------------------------------------------------- the plain forms

def _cache_state(s):
    """The cache's codes, as the numbers that they are in units of their block's scale, and the scales."""
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _places(s, req, pos):
    """Page, slot in it and block in it of positions."""
    page, block = s["case"]["page"], s["case"]["block"]
    slot = pos % page
    return s["table"].long()[req, pos // page], slot, slot // block


def _row_places(s):
    """Request and position of every row."""
    row = torch.arange(s["rows"], device=DEV)
    req = torch.searchsorted(s["row_start"][1:].long(), row, right=True)
    return req, s["ctx"].long()[req] + row - s["row_start"].long()[req]


def _held_places(s):
    """The positions that are cached already in the blocks that requests go on with."""
    block, ctx = s["case"]["block"], s["ctx"].long()
    pos = (ctx // block * block)[:, None] + torch.arange(block, device=DEV)
    return torch.nonzero((pos < ctx[:, None]) & (s["count"] > 0)[:, None], as_tuple=True)[0], pos[
        (pos < ctx[:, None]) & (s["count"] > 0)[:, None]]


def _plain_append(s):
    c = s["case"]
    kind, top, fraction, exponent = FORMATS[c["fmt"]]
    req, pos = _row_places(s)
    held_req, held_pos = _held_places(s)
    page, slot, block = (torch.cat(x) for x in zip(_places(s, held_req, held_pos), _places(s, req, pos)))
    held = held_req.numel()
    for name in ("k", "v"):
        codes, scale = s[name + "_cache"], s[name + "_scale"]
        old = codes.view(torch.int8)[page[:held], slot[:held]].view(kind).float() * scale[page[:held], block[:held]][
            ..., None]
        x = torch.cat([old, s[name].float()])
        shape = (codes.shape[0], c["page"] // c["block"], c["hkv"])
        flat = page * shape[1] + block
        most = torch.zeros((shape[0] * shape[1], c["hkv"]), device=DEV)
        most.scatter_reduce_(0, flat[:, None].expand(-1, c["hkv"]), x.abs().amax(-1), "amax")
        f, e = torch.frexp(most)
        e = torch.where(most > 0, e - exponent + (f > fraction), -126).clamp(min=-126)
        size = torch.ldexp(torch.ones_like(most), e)[flat]
        y = (x / size[..., None]).clamp(-top, top)
        y = (y.round() if c["fmt"] == "i8" else y).to(kind)
        codes.view(torch.int8)[page, slot] = y.view(torch.int8)
        scale[page, block] = size
    return _cache_state(s)


def _plain_read(s):
    page, slot, block = _places(s, *_row_places(s))
    dt, kind = DTYPES[s["case"]["dtype"]], FORMATS[s["case"]["fmt"]][0]
    return {n: (s[n + "_cache"].view(torch.int8)[page, slot].view(kind).float()
                * s[n + "_scale"][page, block][..., None]).to(dt) for n in ("k", "v")}


def _plain_attn(s):
    c, rows, req = s["case"], s["rows"], s["case"]["req"]
    hkv, group, d, width = c["hkv"], c["hq"] // c["hkv"], c["d"], c["n"]
    kind, start = FORMATS[c["fmt"]][0], s["row_start"].long()
    count, ctx = start[1:] - start[:-1], s["ctx"].long()
    # keys and values of every request, padded to the longest
    col = torch.arange(s["longest"], device=DEV)
    live = col < (ctx + count)[:, None]
    page, slot, block = _places(s, torch.arange(req, device=DEV)[:, None], col.expand(req, -1))
    page = page.clamp(min=0)
    k, v = ((s[n + "_cache"].view(torch.int8)[page, slot].view(kind).float() * s[n + "_scale"][page, block][..., None])
            .mul_(live[:, :, None, None]) for n in ("k", "v"))
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


def _plain_verify(s):
    c, n, rows = s["case"], s["case"]["n"], s["rows"]
    start, count = s["row_start"].long(), s["count"].long()
    if rows == 0:
        none = torch.full((c["req"],), -1, dtype=torch.int32, device=DEV)
        return {"accepted": none + 1, "path": s["path"], "next_token": none}
    greedy = c["mode"] == "greedy"
    logits = s["logits"].float()
    i = torch.arange(n, device=DEV)
    live = i < count[:, None]
    at = (start[:-1, None] + i).clamp(max=rows - 1)
    parent = (i - 1).expand(c["req"], -1) if s["parents"] is None else s["parents"].long()[at]
    parent = torch.where(live & (i > 0), parent, -1)
    above = (start[:-1, None] + parent.clamp(min=0)).clamp(max=rows - 1)
    token = torch.where(live, s["tokens"].long()[at], -1)
    # is a row's token taken, if its turn comes (the siblings before it rejected)?
    sibling = (parent[:, :, None] == parent[:, None, :]) & (parent >= 0)[:, :, None] & (i[None, :] < i[:, None])
    same = sibling & (token[:, :, None] == token[:, None, :])
    fits = (parent >= 0) & (token >= 0)
    if greedy:
        best = logits.argmax(-1)
        take = fits & (token == best[above])
    else:
        sharp = float(np.float32(1.0 / c["temp"]))
        top = logits.amax(-1)
        total = torch.exp((logits - top[:, None]) * sharp).sum(-1, dtype=torch.float64)
        # (the few that decide, in 64 bits from the logits on)
        p = torch.exp((logits[above, token.clamp(min=0)].double() - top.double()[above]) * sharp) / total[above]
        p = torch.where(fits & ~same.any(-1), p, 0)
        u = s["uniform"].double()[at]
        if s["draft_probs"] is None:
            take = (p > 0) & (u * (1 - (sibling * p[:, None, :]).sum(-1)) < p)
        else:
            take = fits & (u * s["draft_probs"][at, token.clamp(min=0)].double() < p)
    take = take & ~(sibling & take[:, None, :]).any(-1)  # the first of them
    # a row is on the path where it and all rows above it are taken
    one = ((parent[:, :, None] == i) | torch.eye(n, device=DEV, dtype=torch.bool)).double()
    above_all = torch.linalg.matrix_power(one, 64) > 0
    on = live & ((take | (i == 0))[:, None, :] | ~above_all).all(-1)
    depth = above_all.sum(-1) - 1
    accepted = on.sum(-1) - (count > 0).long()
    last = torch.where(on, i, 0).amax(-1)
    path = s["path"].clone()
    order = torch.full((c["req"], n + 1), -1, dtype=torch.long, device=DEV)
    order.scatter_(1, torch.where(on, depth, n), torch.where(on, i, -1))
    path[at[live]] = order[:, :n][live].int()
    # the token behind the last row that stands
    end = (start[:-1] + last).clamp(max=rows - 1)
    if greedy:
        follow = best[end]
    else:
        mass = torch.exp((logits[end].double() - top[end].double()[:, None]) * sharp) / total[end][:, None]
        if s["draft_probs"] is None:
            child = parent == last[:, None]
            rest = mass.scatter_reduce(1, token.clamp(min=0), torch.where(child & (token >= 0), 0.0, 2.0).double(), "amin")
        else:
            child = (start[:-1] + last + 1).clamp(max=rows - 1)
            more = (last + 1 < count) & (s["tokens"][child] >= 0)
            rest = torch.where(more[:, None], mass - s["draft_probs"][child].double(), mass).clamp(min=0)
        race = s["noise"].double()
        rest = torch.where((rest > 0).any(-1, keepdim=True), rest, mass)
        follow = (rest / race).argmax(-1)
    follow = torch.where((count > 0) & (logits[end].amax(-1) > -math.inf), follow, -1)
    return {"accepted": accepted.int(), "path": path, "next_token": follow.int()}


def run(state):
    if own:
        return _run_own(state)
    return {"append": _plain_append, "read": _plain_read, "attn": _plain_attn, "verify": _plain_verify}[
        state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _values(s, name):
    """The values that the whole cache stands for, [page][slot][head][d]."""
    scale = s[name + "_scale"].double().repeat_interleave(s["case"]["block"], 1)
    return s[name + "_cache"].to(torch.float32).double() * scale[..., None]


def _exact_append(s):
    """Codes before they are rounded, and scales; request after request, block after block."""
    c = s["case"]
    kind, top, _, _ = FORMATS[c["fmt"]]
    if c["req"] * (2 + c["n"] // c["block"]) > 20000:
        return None
    out = {}
    ctx, start, table = s["ctx"].tolist(), s["row_start"].tolist(), s["table"].tolist()
    for name in ("k", "v"):
        codes, scale = s[name + "_cache"].to(torch.float32).double(), s[name + "_scale"].double()
        for b in range(c["req"]):
            end = ctx[b] + start[b + 1] - start[b]
            for at in range(ctx[b] // c["block"] * c["block"], end, c["block"]):
                if end == ctx[b]:
                    continue
                page, slot = table[b][at // c["page"]], at % c["page"]
                held, new = max(0, min(c["block"], ctx[b] - at)), min(c["block"], end - at)
                x = codes[page, slot:slot + new] * scale[page, slot // c["block"]][None, :, None]
                r = start[b] + at - ctx[b]
                x[held:] = s[name][r + held:r + new].double()
                least = x.abs().amax((0, 2)) / top
                size = torch.exp2(torch.log2(least).clamp(min=-126).floor())  # or one above: the logarithm is rounded
                for _ in range(2):
                    size = torch.where(size < least, 2 * size, size)
                size = torch.where(size / 2 >= least, (size / 2).clamp(min=2.0 ** -126), size)
                codes[page, slot:slot + new] = x / size[None, :, None]
                scale[page, slot // c["block"]] = size
        out[name + "_cache"], out[name + "_scale"] = codes if c["fmt"] == "e4m3" else None, scale
    return out


def _exact_read(s):
    out = {}
    ctx, start = s["ctx"].tolist(), s["row_start"].tolist()
    for name in ("k", "v"):
        values = _values(s, name)
        part = []
        for b in range(s["case"]["req"]):
            pos = torch.arange(ctx[b], ctx[b] + start[b + 1] - start[b], device=DEV)
            part.append(values[s["table"][b].long()[pos // s["case"]["page"]], pos % s["case"]["page"]])
        out[name] = torch.cat(part)
    return out


def _exact_attn(s):
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
        page, slot = s["table"][b].long()[position // c["page"]], position % c["page"]
        for h in range(c["hkv"]):
            k, v = (s[m + "_cache"].transpose(1, 2)[:, h].view(torch.int8)[page, slot].view(FORMATS[c["fmt"]][0])
                    .float().double() * s[m + "_scale"][page, slot // c["block"], h].double()[:, None]
                    for m in ("k", "v"))
            for g in range(h * group, (h + 1) * group):
                x = (s["q"][r0:r1, g].double() @ k.T * s["scale"]).masked_fill(~seen, -math.inf)
                lse[r0:r1, g] = torch.logsumexp(x, -1)
                out[r0:r1, g] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers: compared as they are
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attn}[case["op"]](s)
