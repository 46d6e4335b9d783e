"""Rounds over the 8-bit cache end to end: codes and scales after every append as defined, the attended rows against
softmax attention in 64 bits over them, the verdicts against the definition, the contexts read back."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from cache8_helpers import FORMATS, Tree8Case
from round_ops_helpers import DEV
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
