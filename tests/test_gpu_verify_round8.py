"""Rounds over the 8-bit cache end to end: codes and scales after every append as defined, the attended rows against
softmax attention in 64 bits over them, the verdicts against the definition, the contexts read back."""
import importlib.util
import math
import os
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from cache8_helpers import FORMATS, Cache8, Tree8Case
from round_ops_helpers import DEV
from test_gpu_cache8 import append, rows_of
from test_gpu_verify_drafts import VerifyCase

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("verify_round8", os.path.join(ROOT, "examples", "verify_round8.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("inv", [math.inf, 0.25])
def test_rounds_end_to_end(fmt, inv):
    ex = example()
    rng = np.random.default_rng(2)
    phrase = rng.integers(0, ex.VOCAB, 5).tolist()
    prompts = [phrase * 6, rng.integers(0, ex.VOCAB, 17).tolist(), [3] + phrase * 3]
    texts, _ = run(ex, fmt, inv, prompts)
    _, stood = run(ex, fmt, inv, [t + [p[-1]] for p, t in zip(prompts, texts)])
    assert stood > 0 or inv < math.inf  # (the drafts are what the same token was followed by)


def run(ex, fmt, inv, prompts):
    layer = ex.Layer8(requests=3, fmt=FORMATS[fmt][0])
    try:
        texts, ctx, seen = ex.decode(layer, prompts, rounds=6, inv_temperature=inv)
        assert int(layer.status.item()) == 0
        # the cache as it should be, round after round
        c = object.__new__(Tree8Case)
        c.hq, c.hkv, c.d, c.page, c.block, c.fmt = ex.Q_HEADS, ex.KV_HEADS, ex.HEAD_DIM, ex.PAGE, ex.BLOCK, fmt
        c.code, c.kind, c.top = FORMATS[fmt]
        c.n_pages, c.width = layer.n_pages, layer.width
        c.k, c.v = (torch.zeros_like(x).view(c.kind) for x in layer.codes)
        c.k_scale, c.v_scale = (torch.zeros_like(x) for x in layer.scales)
        c.table = layer.table.cpu().numpy().astype(np.int64)  # (pages are only ever added)
        c.dt, c.scale, c.mask = torch.bfloat16, ex.HEAD_DIM ** -0.5, None
        stood = 0
        for step in seen:
            c.start = step["rows"].start.cpu().numpy().astype(np.int64)
            c.ctx, c.counts = step["ctx"], np.diff(c.start).tolist()
            want = c.appended({"k": step["staged"][0], "v": step["staged"][1]})
            for name in ("k", "v"):
                c.raw(name).copy_(torch.from_numpy(want[name]).to(DEV))
                getattr(c, name + "_scale").copy_(torch.from_numpy(want[name + "_scale"]).to(DEV))
            if "q" not in step:
                continue
            c.q = step["q"]
            lse = torch.full(c.q.shape[:2], float("nan"), device=DEV)
            for b in range(3):  # (the example takes no lse: the expected one in its place)
                r0, r1 = int(c.start[b]), int(c.start[b + 1])
                k = c.values("k", b, np.arange(c.ctx[b] + r1 - r0))
                for h in range(c.hq):
                    s = c.q[r0:r1, h].double() @ k[:, h // (c.hq // c.hkv)].T * c.scale
                    lse[r0:r1, h] = torch.logsumexp(torch.where(c.seen(b), s, -math.inf), -1).float()
            c.check(step["attended"], lse)
            v = object.__new__(VerifyCase)
            v.counts, v.start, v.rows, v.vocab = c.counts, c.start, int(c.start[-1]), ex.VOCAB
            v.mode, v.inv, v.q = "greedy" if inv == math.inf else "lookup", inv, None
            v.parents = np.concatenate([np.arange(n) - 1 for n in c.counts])
            v.tokens, v.x, v.u, v.noise = np.array(sum(step["chains"], [])), step["logits"], step["uniform"], step["noise"]
            for got, expected in zip((step["accepted"], step["path"], step["follow"]), v.plain()):
                np.testing.assert_array_equal(got.cpu().numpy(), expected)
            stood += int(step["accepted"].sum())
        for name, codes, scale in (("k", layer.codes[0], layer.scales[0]), ("v", layer.codes[1], layer.scales[1])):
            assert torch.equal(c.raw(name), codes) and torch.equal(getattr(c, name + "_scale"), scale)
        keys, values = layer.read(ctx)
        at = 0
        for b, n in enumerate(ctx):
            for name, got in (("k", keys), ("v", values)):
                assert torch.equal(got[at:at + n], c.values(name, b, np.arange(n)).float().bfloat16())
            at += n
        assert [len(t) for t in texts] == [n + 1 for n in ctx]
        return texts, stood
    finally:
        layer.close()


def test_example_runs():
    example().main()


def test_two_threads_on_streams_of_their_own():
    ex = example()
    rng = np.random.default_rng(5)
    prompts = [[rng.integers(0, ex.VOCAB, n).tolist() * 2 for n in sizes] for sizes in ((40, 9), (3, 60))]

    def one(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            layer = ex.Layer8(requests=2)
            try:
                texts, ctx, seen = ex.decode(layer, prompts[i], rounds=8, inv_temperature=0.5, seed=i)
                out = [texts, ctx, int(layer.status.item())], [s["attended"].clone() for s in seen[1:]], layer.read(ctx)
                torch.cuda.current_stream().synchronize()
                return out
            finally:
                layer.close()

    alone = [one(0), one(1)]
    with ThreadPoolExecutor(2) as pool:
        both = list(pool.map(one, (0, 1)))
    for a, b in zip(alone, both):
        assert a[0] == b[0] and a[0][2] == 0
        assert all(torch.equal(x, y) for x, y in zip(a[1], b[1])) and all(torch.equal(x, y) for x, y in zip(a[2], b[2]))


def test_a_captured_round():
    """Append, attention and verification in one graph, replayed with other rows, lengths and pages: the same bits as call by call."""
    ex = example()
    layers = [ex.Layer8(requests=2) for _ in range(2)]
    try:
        gen = torch.Generator(device=DEV).manual_seed(3)
        for layer in layers:
            prompt = layer.map_rows([0, 0], [49, 6])
            layer.cache_rows8(layer.embed[torch.arange(49 + 6, device=DEV)], prompt, [0, 0])
        # what a round reads, in places that stay
        counts = [3, 2]
        n, heads, d = sum(counts), ex.KV_HEADS, ex.HEAD_DIM
        q = torch.empty((n, ex.Q_HEADS, d), dtype=torch.bfloat16, device=DEV)
        k, v = (torch.empty((n, heads, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        logits = torch.empty((n, ex.VOCAB), dtype=torch.bfloat16, device=DEV)
        tokens, u = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(n, device=DEV)
        noise = torch.empty((2, ex.VOCAB), device=DEV)
        ctx, start = (torch.empty(m, dtype=torch.int32, device=DEV) for m in (2, 3))

        def calls(layer, keep):
            a8 = layer.rows_args(k, v, start, ctx, n)
            out = torch.empty_like(q)
            att = mv.make_tree_attention8_args(
                n_req=2, n_rows=n, max_tree=4, q_heads=ex.Q_HEADS, kv_heads=heads, head_dim=d, dtype=mv.MOE_BF16, q=q.data_ptr(),
                q_stride=q.stride(0), out=out.data_ptr(), out_stride=out.stride(0), row_start=start.data_ptr(), ctx_len=ctx.data_ptr(),
                block_table=layer.table.data_ptr(), table_width=layer.width, cache=layer.cache8(), scale=d ** -0.5,
                dev_status=layer.status.data_ptr())
            acc, follow = (torch.empty(2, dtype=torch.int32, device=DEV) for _ in range(2))
            path = torch.empty(n, dtype=torch.int32, device=DEV)
            ver = mv.make_verify_args(
                n_req=2, n_rows=n, vocab=ex.VOCAB, dtype=mv.MOE_BF16, logits=logits.data_ptr(), stride=logits.stride(0),
                row_start=start.data_ptr(), tokens=tokens.data_ptr(), uniform=u.data_ptr(), noise=noise.data_ptr(),
                noise_stride=noise.stride(0), inv_temperature=1.0, accepted=acc.data_ptr(), path=path.data_ptr(),
                next_token=follow.data_ptr(), dev_status=layer.status.data_ptr())
            ws = [torch.zeros(b, dtype=torch.uint8, device=DEV)
                  for b in (mv.moe_tree_attention8_workspace_bytes(att), mv.moe_verify_drafts_workspace_bytes(ver))]
            keep += [a8, att, ver, ws, out, acc, path, follow]

            def run():
                st = torch.cuda.current_stream().cuda_stream
                mv.moe_cache8_append(a8, st)
                mv.moe_tree_attention8(att, ws[0].data_ptr(), ws[0].numel(), st)
                mv.moe_verify_drafts(ver, ws[1].data_ptr(), ws[1].numel(), st)
            return run, (out, acc, path, follow)

        def fill(at, shape):
            for x in (q, k, v, logits):
                x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
            u.copy_(torch.rand(n, generator=gen, device=DEV))
            noise.exponential_(generator=gen)
            tokens.copy_(torch.randint(0, ex.VOCAB, (n,), generator=gen, device=DEV, dtype=torch.int32))
            ctx.copy_(torch.tensor(at, dtype=torch.int32))
            start.copy_(torch.tensor(np.concatenate([[0], np.cumsum(shape)]), dtype=torch.int32))
            for layer in layers:
                layer.map_rows(at, shape)

        keep = []
        eager, eager_out = calls(layers[0], keep)
        inner, graph_out = calls(layers[1], keep)
        fill([49, 6], [3, 2])
        eager()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            inner()
        for step, (at, shape) in enumerate((([49, 6], [3, 2]), ([51, 8], [1, 4]), ([52, 9], [4, 0]), ([56, 9], [2, 3]))):
            if step:
                fill(at, shape)
                eager()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(eager_out, graph_out)), step
            assert all(torch.equal(x, y) for x, y in zip(layers[0].codes + layers[0].scales, layers[1].codes + layers[1].scales)), step
        assert all(int(layer.status.item()) == 0 for layer in layers)
    finally:
        for layer in layers:
            layer.close()


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_after_a_tree_the_rows_that_stand_are_appended_again(fmt):
    """A tree's rows lie in the cache in their own order: those of its path, gathered from the round's rows, are appended
    once more behind the same context, and the cache is as if the others had only left their scales' rounding."""
    case = Cache8(25, [21, 8, 40], [7, 5, 1], hkv=2, d=64, page=16, block=8, fmt=fmt)
    rows = rows_of(case)
    want = case.appended(rows)
    assert append(case, rows) == 0
    case.same(want)
    trees = VerifyCase(26, case.counts, 500, mode="greedy", tree=True)
    best = trees.x.float().argmax(-1).cpu().numpy()
    for b, n in enumerate(case.counts):  # every second row carries the token that its parent's logits say
        for i in range(1, n):
            r = int(trees.start[b]) + i
            up = int(trees.parents[r])
            trees.tokens[r] = best[trees.start[b] + up] if i % 2 == 0 and up >= 0 else -1
    outs, flags = trees.run()
    assert flags == 0
    for got, expected in zip(outs, trees.plain()):
        np.testing.assert_array_equal(got, expected)
    accepted, path, _ = outs
    assert accepted.max() > 0
    stand = [trees.start[b] + path[trees.start[b]:trees.start[b] + accepted[b] + 1] for b in range(3)]
    at = torch.from_numpy(np.concatenate(stand)).to(DEV)
    assert (np.diff(stand[0]) > 1).any() or (np.diff(stand[1]) > 1).any()  # (something has to move)
    case.counts = [len(s) for s in stand]
    case.start = np.concatenate([[0], np.cumsum(case.counts)])
    rows = {m: x[at] for m, x in rows.items()}
    want = case.appended(rows)
    assert append(case, rows) == 0
    case.same(want)
    for b, n in enumerate(case.counts):
        r0, pos = int(case.start[b]), np.arange(case.ctx[b], case.ctx[b] + n)
        p, o = case.where(b, pos)
        for name in ("k", "v"):
            x, scale = rows[name][r0:r0 + n].double(), getattr(case, name + "_scale")[p, o // 8].double()[..., None]
            step = torch.maximum(x.abs() * 2**-4, scale * 2**-10) if fmt == "e4m3" else scale / 2
            assert ((case.values(name, b, pos) - x).abs() <= step).all()


def test_prompts_of_one_token():
    """Nothing is cached before the first round."""
    ex = example()
    layer = ex.Layer8(requests=2)
    try:
        texts, ctx, _ = ex.decode(layer, [[5], [7]], rounds=3, inv_temperature=math.inf)
        assert int(layer.status.item()) == 0 and [len(t) for t in texts] == [c + 1 for c in ctx] and min(ctx) >= 3
    finally:
        layer.close()
