"""The verify-round example end to end: the attended rows against dense attention in 64 bits over the same
projections (no pages, no cache), the scores against the logits they came from."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from round_ops_helpers import rotate64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("verify_round", os.path.join(ROOT, "examples", "verify_round.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_round_end_to_end():
    ex = example()
    layer = ex.Layer(requests=3)
    try:
        rng = np.random.default_rng(1)
        prompts = [rng.integers(0, ex.VOCAB, n).tolist() for n in (41, 1, 64)]
        drafts = [rng.integers(0, ex.VOCAB, n).tolist() for n in (7, 4, 5)]
        parents = [[-1, 0, 1, 1, 0, 4, -1], [-1, 0, 1, 2], [-1, -1, 0, 0, 3]]
        r = ex.verify_round(layer, prompts, drafts, parents)
        assert r["status"] == 0
        hq, hkv, d = ex.Q_HEADS, ex.KV_HEADS, ex.HEAD_DIM
        rotated = {}
        for name in ("prompt", "rows"):
            qkv = r["prompt_qkv" if name == "prompt" else "qkv"]
            rotated[name] = [rotate64(x, g, r[name].pos, layer.inv_freq, d, False, 1e-6, 1.0)[0]
                             for x, g in ((qkv[:, :hq], layer.q_gain), (qkv[:, hq:hq + hkv], layer.k_gain))]
        p0 = r0 = 0
        for p, t, up in zip(prompts, drafts, parents):
            depth, lines = [], []
            for i, u in enumerate(up):
                depth.append(0 if u < 0 else depth[u] + 1)
                lines.append([i] if u < 0 else lines[u] + [i])
            n, m = len(t), len(p)
            assert r["rows"].pos[r0:r0 + n].tolist() == [m + x for x in depth]
            # keys and values as they are cached: rounded once
            k = torch.cat([rotated["prompt"][1][p0:p0 + m], rotated["rows"][1][r0:r0 + n]]).bfloat16().double()
            v = torch.cat([r["prompt_qkv"][p0:p0 + m, hq + hkv:], r["qkv"][r0:r0 + n, hq + hkv:]]).double()
            q = rotated["rows"][0][r0:r0 + n].bfloat16().double()
            for i in range(n):
                see = list(range(m)) + [m + j for j in lines[i]]
                for h in range(hq):
                    kk, vv = k[see, h // (hq // hkv)], v[see, h // (hq // hkv)]
                    w = torch.softmax(kk @ q[i, h] * d ** -0.5, 0)
                    # three bf16 roundings of the operands may fall the other way (the reference rounds the exact
                    # values, the kernel its own): a step of q and k moves a score by up to 2^-8 of sum |q k|
                    ds = 2 * 2**-8 * d ** -0.5 * float((kk.abs() @ q[i, h].abs()).max())
                    bound = (w[:, None] * vv.abs()).sum(0) * (2 * 2**-8 + 2 * ds) + 2**-8 * (w @ vv).abs()
                    assert ((r["attended"][r0 + i, h].double() - w @ vv).abs() <= bound).all()
            p0, r0 = p0 + m, r0 + n
        logp, entropy, rank, top_ids, top_logp = r["scores"]
        z = torch.log_softmax(r["logits"][r["under"]].double(), -1)
        tok = r["tokens"].long()[torch.from_numpy(r["child"]).to(z.device)]
        own = z.gather(1, tok[:, None])[:, 0]
        assert (logp.double() - own).abs().max() <= 4e-6 + 4e-7 * own.abs().max()
        assert (entropy.double() + (z.exp() * z).sum(-1)).abs().max() <= 1e-4
        assert torch.equal(top_logp, top_logp.sort(-1, descending=True).values)
        assert torch.equal(z.gather(1, top_ids.long()).argmax(-1), torch.zeros_like(tok))
        assert ((rank == 0) == (top_ids[:, 0] == tok)).all()
    finally:
        layer.close()


def test_example_runs():
    example().main()
