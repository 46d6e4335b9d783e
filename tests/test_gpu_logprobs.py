"""moe_token_logprobs against 64 bits; ids and ranks exactly.

Bounds: a log probability is two 32-bit differences and the logarithm of a sum: each term 2^u is off by at most
(|u| + 3) * 2^-23 of itself (u one subtraction, one product, the exponential 2^-22), weighted by its share p the mean of
|u| stays below 24 (p |log2 p| of 2^24 entries), so log s is off by under 4e-6; the differences add 2^-23 of their
value.  4e-6 + 4e-7 |value|.  The entropy adds sum p |u| errors: 4e-6 + 4e-6 |value|, on both of its parts.
"""
import math

import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from round_ops_helpers import DEV, DT, TreeCase, at, stream, word

pytestmark = pytest.mark.gpu


def run(x, token, k, inv_t=1.0, stride=None, times=1, want=("logp", "entropy", "rank")):
    code = {torch.bfloat16: mv.MOE_BF16, torch.float16: mv.MOE_F16, torch.float32: mv.MOE_F32}[x.dtype]
    rows, vocab = x.shape
    f = lambda *s: torch.full(s, 9.0, device=DEV)  # noqa: E731
    o = dict(logp=f(rows), entropy=f(rows), rank=torch.full((rows,), -9, dtype=torch.int32, device=DEV),
             top_ids=torch.full((rows, k), -9, dtype=torch.int32, device=DEV), top_logp=f(rows, k))
    status = word()
    args = mv.make_logprob_args(
        n_rows=rows, vocab=vocab, dtype=code, logits=at(x), stride=x.stride(0) if stride is None else stride,
        dev_status=at(status), tokens=at(token), top_k=k, inv_temperature=inv_t, top_ids=at(o["top_ids"]) if k else 0,
        top_logp=at(o["top_logp"]) if k else 0, **{n: at(o[n]) for n in want})
    ws = torch.zeros(mv.moe_token_logprobs_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    for _ in range(times):
        mv.moe_token_logprobs(args, at(ws), ws.numel(), stream())
    return o, int(status.item())


def check(x, token, k, inv_t=1.0, **kw):
    o, status = run(x, token, k, inv_t, **kw)
    assert status == 0
    inv = float(np.float32(inv_t))
    xs, tok = x.float().cpu().numpy(), token.cpu().numpy()
    for r in range(x.shape[0]):
        z = xs[r].astype(np.float64) * inv
        order = np.lexsort((np.arange(z.size), -xs[r]))
        live = z > -np.inf
        if live.any():
            m = z.max()
            lp = (z - m) - math.log(np.exp(z[live] - m).sum())  # m apart: it may be as large as the type's
            ent = -(np.exp(lp[live]) * lp[live]).sum()
        else:
            lp, ent = np.full(z.size, -np.inf), 0.0
        got = float(o["logp"][r])
        ref = lp[tok[r]] if 0 <= tok[r] else -np.inf
        assert got == ref or abs(got - ref) <= 4e-6 + 4e-7 * abs(ref), (r, got, ref)
        got = float(o["entropy"][r])
        spread = abs(lp[order[0]]) + abs(ent) if live.any() else 0.0
        assert abs(got - ent) <= 4e-6 + 4e-6 * spread, (r, got, ent)
        if 0 <= tok[r]:
            assert int(o["rank"][r]) == int(np.nonzero(order == tok[r])[0][0])
        else:
            assert int(o["rank"][r]) == -1
        n = min(k, int(live.sum()))
        ids, lps = o["top_ids"][r].cpu().numpy(), o["top_logp"][r].cpu().numpy()
        np.testing.assert_array_equal(ids[:n], order[:n])
        assert (ids[n:] == -1).all() and (lps[n:] == -np.inf).all()
        assert (np.abs(lps[:n] - lp[order[:n]]) <= 4e-6 + 4e-7 * np.abs(lp[order[:n]])).all()
    return o


def sample(seed, rows, vocab, dtype, spread=2.5):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn((rows, vocab), generator=gen, device=DEV) * spread).to(DT[dtype][0])
    return x, torch.randint(0, vocab, (rows,), generator=gen, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 5, 31, 33, 1000, 8191, 8193, 32003, 131072])
@pytest.mark.parametrize("rows,k", [(1, 20), (3, 32), (16, 1), (40, 5), (2, 0)])
def test_logprobs(dtype, vocab, rows, k):
    x, t = sample(vocab + rows, rows, vocab, dtype)
    check(x, t, k, 0.8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(dtype):
    x, t = sample(1, 700, 4099, dtype)
    check(x, t, 8)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_any_alignment_and_stride(dtype):
    """Columns 1.. and 3.. of a wider buffer of odd width: rows start anywhere in a 16-byte vector."""
    wide, t = sample(2, 9, 20011, dtype)
    for first, last in ((1, 20011), (3, 20000), (5, 12), (20010, 20011)):
        x = wide[:, first:last]
        check(x, (t % (last - first)).to(torch.int32), min(3, 32), stride=wide.stride(0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["equal", "rising", "falling", "few", "steps"])
def test_orders_and_ties(dtype, order):
    vocab = 40001
    i = torch.arange(vocab, device=DEV, dtype=torch.float32)
    row = {"equal": torch.zeros_like(i), "rising": i / 5000, "falling": -i / 5000, "few": torch.floor(i / 100) % 3,
           "steps": torch.floor(-i / 4096)}[order]
    x = row.to(DT[dtype][0]).repeat(2, 1)
    t = torch.tensor([0, vocab - 1], dtype=torch.int32, device=DEV)
    for k in (1, 20, 32):
        check(x, t, k)


def test_signed_zeros_tie():
    x = torch.zeros((1, 5000), device=DEV)
    x[0, ::2] = -0.0
    check(x, torch.tensor([17], dtype=torch.int32, device=DEV), 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masked_entries(dtype):
    x, t = sample(3, 8, 9001, dtype)
    x[0, :] = -float("inf")
    x[1, :] = -float("inf")
    x[1, 4000] = 1.0
    x[2, 7:] = -float("inf")
    x[3, ::2] = -float("inf")
    x[4, 5] = torch.finfo(x.dtype).min
    x[5, :] = torch.finfo(x.dtype).min
    t[:6] = torch.tensor([3, 4000, 9000, 2, 5, 11], dtype=torch.int32)
    check(x, t, 12)


def test_peaked_rows():
    x, t = sample(4, 4, 50000, "f32")
    x[:, 123] = 60.0
    x[2] *= 1e4
    t[:2] = 123
    check(x, t, 5, 1.3)


def test_tokens_that_are_none_or_outside():
    x, t = sample(5, 4, 3001, "f32")
    t[1] = -1
    check(x, t, 4)
    t[2], t[3] = 3001, -2**31
    o, status = run(x, t, 4)
    assert status == mv.MOE_DEV_INDEX
    assert o["rank"].tolist()[1:] == [-1, -1, -1] and (o["logp"][1:] == -float("inf")).all()


def test_outputs_that_are_not_wanted():
    x, t = sample(6, 3, 5000, "bf16")
    full, _ = run(x, t, 6)
    for want in ((), ("logp",), ("entropy",), ("rank", "entropy")):
        o, status = run(x, t if "logp" in want or "rank" in want else None, 6, want=want)
        assert status == 0
        for n in ("logp", "entropy", "rank"):
            assert torch.equal(o[n], full[n]) == (n in want)
        assert torch.equal(o["top_ids"], full["top_ids"])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_rows_stay_alone(value):
    x, t = sample(7, 5, 30000, "f32")
    clean, _ = run(x, t, 8)
    x[2, 777] = value
    o, _ = run(x, t, 8)
    rest = [0, 1, 3, 4]
    for n, v in o.items():
        assert torch.equal(v[rest], clean[n][rest])
    assert torch.isnan(o["entropy"][2])


def test_zero_rows_and_repeats():
    x, t = sample(8, 0, 100, "f32")
    run(x, t, 4)
    x, t = sample(9, 6, 100003, "bf16")
    a, _ = run(x, t, 20)
    b, _ = run(x, t, 20, times=4)
    for n in a:
        assert torch.equal(a[n], b[n])


def test_captured():
    x, t = sample(10, 3, 60001, "bf16")
    o = dict(logp=torch.zeros(3, device=DEV), rank=torch.zeros(3, dtype=torch.int32, device=DEV))
    status = word()
    args = mv.make_logprob_args(n_rows=3, vocab=60001, dtype=mv.MOE_BF16, logits=at(x), stride=60001,
                                dev_status=at(status), tokens=at(t), logp=at(o["logp"]), rank=at(o["rank"]))
    ws = torch.zeros(mv.moe_token_logprobs_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mv.moe_token_logprobs(args, at(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    for seed in (11, 12):
        y, _ = sample(seed, 3, 60001, "bf16")
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want, _ = run(x, t, 0)
        assert torch.equal(o["logp"], want["logp"]) and torch.equal(o["rank"], want["rank"])


def call(x, token, k, ws):
    """One call over a given workspace; all outputs."""
    code = {torch.bfloat16: mv.MOE_BF16, torch.float16: mv.MOE_F16, torch.float32: mv.MOE_F32}[x.dtype]
    rows, vocab = x.shape
    f = lambda *s: torch.full(s, 9.0, device=DEV)  # noqa: E731
    o = dict(logp=f(rows), entropy=f(rows), rank=torch.full((rows,), -9, dtype=torch.int32, device=DEV),
             top_ids=torch.full((rows, k), -9, dtype=torch.int32, device=DEV), top_logp=f(rows, k))
    status = word()
    args = mv.make_logprob_args(n_rows=rows, vocab=vocab, dtype=code, logits=at(x), stride=x.stride(0),
                                dev_status=at(status), tokens=at(token), top_k=k, **{n: at(t) for n, t in o.items()})
    mv.moe_token_logprobs(args, at(ws), ws.numel(), stream())
    assert int(status.item()) == 0
    return o


SHAPES = [(16, 131072, 20, "bf16"), (100, 32003, 5, "f32"), (5, 60001, 32, "f32"), (140, 40000, 3, "f32"),
          (1, 262144, 1, "f16"), (152, 33000, 8, "f32"), (200, 9001, 4, "bf16"), (16, 131072, 20, "bf16"),
          (77, 131072, 2, "bf16"), (152, 33000, 8, "f32")]


def test_one_workspace_serves_calls_of_any_shape():
    """Set to zero once, then used by rounds of other row counts, vocabularies and list lengths."""
    inputs = [sample(20 + i, rows, vocab, dtype) + (k,) for i, (rows, vocab, k, dtype) in enumerate(SHAPES)]
    size = max(mv.moe_token_logprobs_workspace_bytes(mv.make_logprob_args(
        n_rows=x.shape[0], vocab=x.shape[1], dtype=DT[shape[3]][1], logits=at(x), stride=x.stride(0), dev_status=at(t),
        tokens=at(t), logp=at(t))) for (x, t, _), shape in zip(inputs, SHAPES))
    shared = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for (x, t, k), shape in zip(inputs, SHAPES):
        want = call(x, t, k, torch.zeros_like(shared))
        got = call(x, t, k, shared)
        for n in want:
            assert torch.equal(got[n], want[n]), (shape, n)


def test_a_workspace_shared_with_the_attention():
    """The attention's and this call's workspaces may be one buffer, as long as the calls do not overlap."""
    case = TreeCase(30, [5000, 12, 700], [16, 3, 30], hq=16, hkv=2, d=128, page=16, dtype="bf16")
    out, lse, status = case.run()
    assert status == 0
    x, t = sample(31, 140, 40000, "f32")
    few, few_t = sample(32, 3, 100000, "bf16")
    o2, l2 = case.outputs()
    flag = word()
    args = case.args(o2, l2, flag)
    shared = torch.zeros(max(1 << 20, mv.moe_tree_attention_workspace_bytes(args)), dtype=torch.uint8, device=DEV)
    want, few_want = (call(a, b, 8, torch.zeros_like(shared)) for a, b in ((x, t), (few, few_t)))
    for _ in range(3):
        o2.fill_(float("nan"))
        mv.moe_tree_attention(args, at(shared), shared.numel(), stream())
        assert int(flag.item()) == 0 and torch.equal(o2, out) and torch.equal(l2, lse)
        for (a, b), w in (((x, t), want), ((few, few_t), few_want)):
            got = call(a, b, 8, shared)
            for n in w:
                assert torch.equal(got[n], w[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab", [(6, 5003), (6, 70001), (162, 9001)])
def test_masks_of_the_lowest_value(dtype, rows, vocab):
    """Masked entries that hold the type's lowest finite number, alone in a thread's part, a warp's, a slice or at
    a row's start: finite logits have finite entropies."""
    x, t = sample(33, rows, vocab, dtype)
    i = torch.arange(vocab, device=DEV)
    masks = [(i != 17) & (i != vocab // 2) & (i != vocab - 3), i < vocab // 2, i >= vocab // 2, i % 2 == 0,
             i // 4096 % 2 == 0, i != vocab - 1]
    for r in range(rows):
        x[r, masks[r % 6]] = torch.finfo(x.dtype).min
    check(x, t, 5)


@pytest.mark.parametrize("inv_t", [1e-30, 1e6, 1e30, 2.3e38, 3e38, 3.4e38])
def test_extreme_temperatures(inv_t):
    """Down to the largest factor that 32 bits hold, where the first entry has all the probability."""
    x, t = sample(34, 4, 20011, "f32")
    t[0], t[1] = x[0].argmax(), x[1].argmax()
    o, status = run(x, t, 2, inv_t)
    assert status == 0
    if inv_t < 1:
        check(x, t, 2, inv_t)
        return
    assert o["logp"].tolist()[:2] == [0.0, 0.0] and (o["logp"][2:] < -1e3).all()
    assert (o["entropy"] == 0).all() and (o["top_logp"][:, 0] == 0).all() and (o["top_logp"][:, 1] < -1e3).all()
    assert torch.equal(o["top_ids"][:, 0].long(), x.argmax(1))
