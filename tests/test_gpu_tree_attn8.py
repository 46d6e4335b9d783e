"""moe_tree_attention8 against softmax attention in 64 bits; the bound of each element is derived in Tree8Case.check.

Up to 32 query rows a key/value head take one kernel, more another: both are met by every kind of test.
"""
import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from cache8_helpers import Tree8Case
from round_ops_helpers import DEV, at, i32, stream, word

pytestmark = pytest.mark.gpu


def good(case, status=0, **kw):
    out, lse, got = case.run()
    assert got == status
    case.check(out, lse, **kw)
    return out, lse


@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("i8", "f16"), ("e4m3", "f16"), ("i8", "bf16")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,n", [(1, 1, 3), (4, 1, 4), (6, 2, 9), (16, 1, 2), (24, 8, 12), (32, 4, 16), (20, 1, 8)])
def test_heads_and_types(fmt, dtype, d, hq, hkv, n):
    good(Tree8Case(d + hq, [0, 5, 130, 64, 63], [n, 1, n, 0, 1], hq=hq, hkv=hkv, d=d, page=16, block=16, fmt=fmt, dtype=dtype))


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 33, 63, 64])
@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
def test_tree_widths_and_masks(n, mask):
    good(Tree8Case(n, [0, 200, 61], [n, n, max(0, n - 1)], hq=8, hkv=2, d=128, page=16, block=8, fmt="e4m3", mask=mask))
    good(Tree8Case(n, [0, 200, 61], [n, n, max(0, n - 1)], hq=2, hkv=2, d=64, page=32, block=16, fmt="i8", mask=mask))


@pytest.mark.parametrize("page,block", [(1, 1), (3, 1), (8, 8), (24, 8), (16, 16), (64, 16), (64, 2), (100, 4), (128, 128), (256, 64)])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("n", [2, 40])
def test_pages_blocks_and_layouts(page, block, layout, n):
    good(Tree8Case(page, [77, 300, 0, 255], [n, 6, 5, 1], hq=6, hkv=3, d=64, page=page, block=block, fmt="i8", dtype="f16", layout=layout))
    good(Tree8Case(page, [77, 300, 0, 255], [n, 6, 5, 1], hq=4, hkv=2, d=128, page=page, block=block, fmt="e4m3", layout=layout))


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 4097])
def test_context_lengths(ctx):
    good(Tree8Case(ctx, [ctx], [5], hq=8, hkv=1, d=128, page=16, block=16, fmt="e4m3"))
    good(Tree8Case(ctx, [ctx], [1], hq=4, hkv=4, d=64, page=16, block=16, fmt="i8", dtype="f16"))
    good(Tree8Case(ctx, [ctx], [1], hq=4, hkv=2, d=256, page=16, block=4, fmt="e4m3"))


@pytest.mark.parametrize("hq,hkv,n,d", [(32, 4, 1, 128), (32, 4, 4, 128), (32, 4, 16, 128), (32, 4, 64, 128), (8, 8, 1, 64), (8, 8, 30, 64),
                                        (16, 1, 64, 128), (64, 1, 40, 128), (128, 2, 3, 64), (16, 2, 2, 256), (16, 2, 33, 256)])
def test_long_contexts_split_over_blocks(hq, hkv, n, d):
    good(Tree8Case(hq + n, [20011], [n], hq=hq, hkv=hkv, d=d, page=64, block=32, fmt="e4m3"))
    good(Tree8Case(hq + n, [9000, 3], [n, 1], hq=hq, hkv=hkv, d=d, page=24, block=8, fmt="i8", dtype="f16", layout="hnd"))


@pytest.mark.parametrize("req,n", [(70, 20), (300, 5), (383, 4), (384, 4), (385, 4), (900, 3), (300, 40)])
def test_ragged_batches_and_more_requests_than_threads(req, n):
    rng = np.random.default_rng(req)
    ctx = rng.integers(0, 300, req)
    ctx[::7] = 0
    counts = rng.integers(0, n + 1, req)
    good(Tree8Case(req, ctx.tolist(), counts.tolist(), hq=8, hkv=2, d=64, page=16, block=16, fmt="e4m3", max_tree=n))


def test_rows_that_see_nothing():
    for hq in (4, 40):
        case = Tree8Case(4, [0, 0, 40], [6, 1, 3], hq=hq, hkv=2, d=64, page=16, block=16, fmt="i8", mask="random")
        case.mask[0] = 0
        case.mask[6] = 0
        out, lse = good(case)
        assert (out[0] == 0).all() and (lse[6] == -float("inf")).all()


def test_all_requests_empty():
    case = Tree8Case(5, [10, 0], [0, 0], hq=4, hkv=2, d=64, page=16, block=16, fmt="e4m3")
    assert case.run()[2] == 0


@pytest.mark.parametrize("n,hq", [(5, 4), (16, 32), (64, 16), (3, 4)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_masked_nan_codes_have_no_influence(n, hq, d):
    """A tree row whose cached codes are NaN changes only the rows that see it, which get NaN where it is."""
    case = Tree8Case(6, [90], [n], hq=hq, hkv=2, d=d, page=16, block=16, fmt="e4m3")
    clean, clean_lse = good(case)
    seen = case.seen(0)[:, 90:]
    j = n // 2
    p, o = case.where(0, np.array([90 + j]))
    case.raw("v")[p, o, :, 3:9] = 0xff
    out, lse, status = case.run()
    assert status == 0
    hit = seen[:, j].cpu()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
    assert torch.isnan(out[hit][:, :, 3:9]).all() and torch.equal(out[hit][:, :, 9:], clean[hit][:, :, 9:])
    case.raw("k")[p, o] = 0x7f
    out, lse, status = case.run()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()


@pytest.mark.parametrize("n", [2, 40])
def test_what_lies_past_the_end_has_no_influence(n):
    case = Tree8Case(7, [45], [n], hq=4, hkv=2, d=128, page=32, block=32, fmt="e4m3")
    clean, clean_lse = good(case)
    end = 45 + n
    page, slot = int(case.table[0, end // 32]), end % 32
    if slot:
        for name in ("k", "v"):
            case.raw(name)[page, slot:] = 0x7f
    out, lse, status = case.run()
    assert status == 0 and torch.equal(out, clean) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("block", [4, 16])
def test_pages_that_are_none(n, block):
    case = Tree8Case(8, [100], [n], hq=4, hkv=2, d=64, page=16, block=block, fmt="e4m3")
    unused = sorted(set(range(case.n_pages)) - set(case.table[0].tolist()))
    case.raw("v")[unused] = 0x7f  # (NaN, in pages of nobody)
    case.table[0, 2] = -1
    case.table[0, 4] = case.n_pages
    hidden = torch.zeros(100 + n, dtype=torch.bool, device=DEV)
    hidden[32:48] = True
    hidden[64:80] = True
    out, lse, status = case.run()
    assert status == mv.MOE_DEV_INDEX
    case.table[0, 2] = case.table[0, 4] = 0  # (read by the check alone, and hidden there)
    case.check(out, lse, hidden=lambda b: hidden)


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("block", [4, 16])
@pytest.mark.parametrize("value,raised", [(0.0, 0), (float("nan"), mv.MOE_DEV_VALUE), (float("inf"), mv.MOE_DEV_VALUE),
                                          (-1.0, mv.MOE_DEV_VALUE), (2.0**-126, 0), (2.0**-60, 0)])
def test_scales_of_zero_and_scales_that_are_none(n, block, value, raised):
    """Such keys and values are zeros (values too where the scale is tiny), and weigh as zeros do."""
    case = Tree8Case(9, [100], [n], hq=4, hkv=2, d=64, page=16, block=block, fmt="e4m3")
    for c in (1, 3):
        page = int(case.table[0, c])
        case.v_scale[page] = value
        if not value > 0 or value == float("inf"):
            case.k_scale[page, 0] = value
    out, lse, status = case.run()
    assert status == raised
    for c in (1, 3):
        page = int(case.table[0, c])
        case.v_scale[page] = 0
        if not value > 0 or value == float("inf"):
            case.k_scale[page, 0] = 0
    case.check(out, lse)


@pytest.mark.parametrize("n", [2, 40])
def test_a_context_of_zero_values(n):
    """An appended block of zeros has the smallest scale; the weights' sum is as with any other."""
    case = Tree8Case(10, [70], [n], hq=4, hkv=1, d=64, page=16, block=16, fmt="i8")
    case.raw("v").zero_()
    case.v_scale.fill_(2.0**-126)
    out, lse, status = case.run()
    assert status == 0 and (out == 0).all()
    case.v_scale.fill_(1)
    case.check(out, lse)


@pytest.mark.parametrize("n", [2, 40])
def test_scales_far_apart(n):
    case = Tree8Case(11, [200], [n], hq=4, hkv=2, d=64, page=16, block=16, fmt="e4m3")
    case.v_scale.mul_(torch.exp2(torch.randint(-20, 20, case.v_scale.shape, device=DEV).float()))
    good(case)


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scores_of_any_size(n, scale):
    good(Tree8Case(12, [300, 7], [n, 3], hq=4, hkv=2, d=64, page=16, block=16, fmt="e4m3", scale=scale))


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("factor", [2.0**-60, 2.0**60])
def test_queries_of_any_size(n, factor):
    """bf16 queries that fp16 does not hold: a row's power of two takes care of it."""
    case = Tree8Case(13, [150], [n], hq=4, hkv=2, d=64, page=16, block=16, fmt="i8")
    case.q = (case.q.float() * factor).to(case.dt)
    case.scale = case.scale / factor
    good(case)


@pytest.mark.parametrize("n", [2, 40])
def test_scores_that_rise_and_fall_in_steps(n):
    """The running maximum moves inside a tile, between tiles and not at all."""
    for seed, steps in ((1, [0, 9, 3, 30, 30, 12, 60]), (2, [60, 40, 20, 0]), (3, [0, 5, 10, 15, 20, 25, 30, 35])):
        case = Tree8Case(seed, [len(steps) * 48], [n], hq=4, hkv=1, d=64, page=16, block=16, fmt="e4m3", mask="chain")
        case.q.fill_(0)
        case.q[:, :, 0] = 8.0
        codes = case.raw("k")
        for i, s in enumerate(steps):
            p, o = case.where(0, np.arange(48 * i, 48 * i + 48))
            value = torch.tensor(float(s), device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[p, o, :, 0] = value
        case.k_scale.fill_(1.0)
        good(case)


def test_strides_padding_and_rows_of_nobody():
    for n in (3, 40):
        case = Tree8Case(14, [50, 9], [n, 2], hq=4, hkv=2, d=64, page=16, block=16, fmt="i8", q_pad=24, pad_rows=5)
        out, lse = good(case)
        assert torch.isnan(out[n + 2:]).all() and torch.isnan(lse[n + 2:]).all()


def test_bad_lengths():
    for hq in (4, 40):
        case = Tree8Case(15, [40, 30, 20, 10], [3, 4, 2, 5], hq=hq, hkv=2, d=64, page=16, block=16, fmt="e4m3", max_tree=4)
        out, lse, status = case.run(ctx=i32([40, -1, 20, 10]))
        assert status == mv.MOE_DEV_LENGTH
        case.check(out, lse, only=[0, 2])
        for rows in (slice(3, 7), slice(9, 14)):  # a negative context; more rows than max_tree
            assert (out[rows] == 0).all() and (lse[rows] == -float("inf")).all()
        out, lse, status = case.run(start=i32([0, 3, 2, 9, 2**31 - 1]))
        assert status & mv.MOE_DEV_LENGTH


def test_bits_do_not_change_from_call_to_call_nor_with_other_rows():
    for hq, n in ((8, 4), (16, 16)):
        case = Tree8Case(16, [3000], [n], hq=hq, hkv=2, d=128, page=16, block=16, fmt="e4m3")
        first = case.run()
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(first[:2], case.run()[:2]))
        case.q[1:] = case.q[1:] * 3  # the other rows' queries
        again = case.run()
        assert torch.equal(first[0][0], again[0][0]) and torch.equal(first[1][0], again[1][0])


def test_one_workspace_for_calls_of_many_shapes():
    """Also of the 16-bit cache's kind and the log probabilities': counters are zero between calls."""
    cases = [Tree8Case(s, [c], [n], hq=hq, hkv=2, d=d, page=16, block=16, fmt="e4m3")
             for s, c, n, hq, d in ((1, 5000, 1, 8, 128), (2, 3000, 40, 16, 128), (3, 2500, 2, 4, 256), (4, 9000, 30, 8, 64))]
    ready = []
    for case in cases:
        out, lse = case.outputs()
        status = word()
        ready.append((case, out, lse, status, case.args(out, lse, status), case.keep))
    ws = torch.zeros(max(mv.moe_tree_attention8_workspace_bytes(r[4]) for r in ready), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        for case, out, lse, status, args, _ in ready:
            mv.moe_tree_attention8(args, at(ws), ws.numel(), stream())
    for case, out, lse, status, _, _ in ready:
        assert int(status.item()) == 0
        case.check(out, lse)


@pytest.mark.parametrize("n", [2, 40])
def test_a_replayed_graph_follows_contents_on_another_stream(n):
    case = Tree8Case(17, [900, 40], [n, 3], hq=4, hkv=2, d=64, page=16, block=16, fmt="i8")
    out, lse = case.outputs()
    status, ctx = word(), i32(case.ctx)
    args = case.args(out, lse, status, ctx=ctx)
    ws = torch.zeros(mv.moe_tree_attention8_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        mv.moe_tree_attention8(args, at(ws), ws.numel(), stream())
    for lengths in ([900, 40], [500, 0], [3, 33]):
        ctx.copy_(i32(lengths))
        graph.replay()
        torch.cuda.synchronize()
        case.ctx = lengths
        case.check(out, lse)
    assert int(status.item()) == 0


@pytest.mark.parametrize("hq", [4, 32])
def test_waits_that_give_up(hq):
    """With a bound of 1 ns waits may give up at once: the call ends and says so, and a clean workspace serves again."""
    case = Tree8Case(18, [30000], [4], hq=hq, hkv=1, d=128, page=64, block=64, fmt="e4m3")
    mv.moe_set_attention_wait_limit_ns(1)
    try:
        _, _, status = case.run()
    finally:
        mv.moe_set_attention_wait_limit_ns(0)
    assert status in (0, mv.MOE_DEV_TIMEOUT)
    good(case)


def test_long_flat_tails_beside_a_strong_key():
    """100,000 keys of weight 2^-17 of the strongest each, together most of the result."""
    for n in (1, 40):
        case = Tree8Case(19, [100000], [n], hq=1, hkv=1, d=64, page=64, block=64, fmt="e4m3", mask="chain", scale=1.0)
        case.raw("k").zero_()
        case.k_scale.fill_(1.0)
        case.q.zero_()
        case.q[:, :, 0] = 1.0
        p, o = case.where(0, np.array([5]))
        case.raw("k")[p, o, :, 0] = torch.tensor(12.0, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
        good(case)


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("block", [4, 8, 16])
@pytest.mark.parametrize("value,raised", [(0.0, 0), (2.0**-60, 0), (float("nan"), mv.MOE_DEV_VALUE), (2.0**60, mv.MOE_DEV_VALUE)])
def test_nan_codes_under_scales_that_count_as_zero(n, block, value, raised):
    """A NaN code is NaN whatever its scale (0 times it, too), in both kernels: for every row in the context, in drafted
    rows for those that see them; other elements are as they are without it."""
    case = Tree8Case(20, [90], [n], hq=4, hkv=2, d=64, page=16, block=block, fmt="e4m3")
    pages = [int(case.table[0, c]) for c in (1, 5)]  # positions 16..31, and 80..95 with drafted rows
    for page in pages:
        case.v_scale[page] = value
    clean, clean_lse, status = case.run()
    assert status == raised and torch.isfinite(clean).all()
    p, o = case.where(0, np.array([90 + 1]))  # a drafted row
    case.raw("v")[p, o, :, 3:9] = 0xff
    out, lse, status = case.run()
    hit = case.seen(0)[:, 91].cpu()
    assert status == raised and hit.any() and torch.equal(lse, clean_lse)
    assert torch.isnan(out[hit][:, :, 3:9]).all() and torch.equal(out[~hit], clean[~hit])
    assert torch.equal(out[hit][:, :, 9:], clean[hit][:, :, 9:]) and torch.equal(out[hit][:, :, :3], clean[hit][:, :, :3])
    p, o = case.where(0, np.array([20]))  # of the context
    case.raw("v")[p, o, 1, 40:42] = 0x7f
    more, lse, status = case.run()
    assert status == raised and torch.equal(lse, clean_lse)
    assert torch.isnan(more[:, 2:, 40:42]).all()
    more[:, 2:, 40:42] = out[:, 2:, 40:42]
    assert torch.equal(torch.nan_to_num(more, nan=99.0), torch.nan_to_num(out, nan=99.0))


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("dtype,largest,small,rounded", [("bf16", 1.0, 2.0**-31 * 1.9921875, False), ("bf16", 1.0, 2.0**-33 * 1.9921875, True),
                                                         ("f16", 40000.0, 2.0**-13 * 1.9990234375, False),
                                                         ("f16", 40000.0, 2.0**-14 * 1.9990234375, True)])
def test_queries_with_elements_far_below_their_largest(n, dtype, largest, small, rounded):
    """As fp16 numbers, with the largest at 2^14 or above: exact from 2^-31 (fp16 queries 2^-28) of the largest on, below
    that off by 2^-25, so 2^-39 of the largest, at most.  Its key is 0, the score comes from the small ones alone."""
    case = Tree8Case(22, [1], [n], hq=4, hkv=2, d=64, page=16, block=16, fmt="e4m3", dtype=dtype, mask="random", scale=2.0**30 / largest)
    case.mask.zero_()  # the rows see the one context position: lse is its score
    case.q.fill_(small)
    case.q[:, :, 0] = largest
    p, o = case.where(0, np.array([0]))
    case.raw("k")[p, o] = 0x38  # 1
    case.raw("k")[p, o, :, 0] = 0
    case.k_scale.fill_(1.0)
    score = 63 * float(case.q[0, 0, 1]) * case.scale
    _, lse, status = case.run()
    assert status == 0
    off = (lse.double() - score).abs().max().item()
    assert off <= 66 * 2**-24 * score + (63 * 2**-39 * largest * case.scale if rounded else 0) + 2**-22 * (score + 48) + 4e-6
    assert off > 66 * 2**-24 * score + 2**-22 * (score + 48) + 4e-6 or not rounded


@pytest.mark.parametrize("hq", [4, 32])
def test_waits_that_give_up_are_reported(hq):
    """Blocks that share a head end at different times, so with a bound of 1 ns some call's wait gives up."""
    case = Tree8Case(23, [30000], [4], hq=hq, hkv=1, d=128, page=64, block=64, fmt="e4m3")
    mv.moe_set_attention_wait_limit_ns(1)
    try:
        seen = [case.run()[2] for _ in range(10)]
    finally:
        mv.moe_set_attention_wait_limit_ns(0)
    assert set(seen) <= {0, mv.MOE_DEV_TIMEOUT} and mv.MOE_DEV_TIMEOUT in seen
    good(case)


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("q,k,scale", [(2.0**100, 2.0**-100, 1 / 8), (2.0**-100, 2.0**100, 1 / 8), (2.0**60, 2.0**60, 2.0**-123),
                                       (2.0**-40, 2.0**-60, 2.0**97), (2.0**20, 2.0**-120, 2.0**97)])
def test_queries_and_scales_far_from_one_whose_scores_are_ordinary(n, q, k, scale):
    case = Tree8Case(24, [150], [n], hq=4, hkv=2, d=64, page=16, block=16, fmt="e4m3", scale=scale)
    case.q = (case.q.float() * q).to(case.dt)
    case.k_scale.mul_(k)  # (at 2^-120 some are no normal numbers: they count as 0, which is said)
    none = case.k_scale < 2.0**-126
    p, _ = case.where(0, np.arange(150 + n))
    out, lse, status = case.run()
    assert status == (mv.MOE_DEV_VALUE if none[p].any() else 0)
    case.k_scale[none] = 0
    case.check(out, lse)


@pytest.mark.parametrize("first", [-2**31, -2**31 + 1, -2**31 + 5, -2**30, -1])
@pytest.mark.parametrize("hq", [4, 40])
def test_row_starts_as_far_below_zero_as_they_go(hq, first):
    """The request that begins there, and the one that ends there, are left out; no row is written for them."""
    case = Tree8Case(25, [40, 30, 20, 10], [3, 4, 2, 5], hq=hq, hkv=2, d=64, page=16, block=16, fmt="e4m3", max_tree=5)
    out, lse, status = case.run(start=i32([0, first, 7, 9, 14]))
    assert status == mv.MOE_DEV_LENGTH
    case.check(out, lse, only=[2, 3])
    assert torch.isnan(out[:7]).all() and torch.isnan(lse[:7]).all()


@pytest.mark.parametrize("n", [2, 40])
def test_one_scale_for_all_by_strides_of_zero(n):
    """A cache under one calibrated scale of keys and one of values: strides of 0, attended and read."""
    case = Tree8Case(26, [150, 20], [n, 1], hq=4, hkv=2, d=64, page=16, block=16, fmt="i8")
    for name, value in (("k", 0.011), ("v", 0.017)):
        setattr(case, name + "_scale", torch.full((1, 1, 1), value, device=DEV).expand(case.n_pages, 1, 2))
    assert case.cache().scale_page_stride == 0 and case.cache().scale_head_stride == 0
    good(case)
    out = torch.empty((n + 1, 4, 64), dtype=torch.float32, device=DEV)
    status = word()
    mv.moe_cache8_read(case.rows_args(out[:, :2], out[:, 2:], status), stream())
    assert int(status.item()) == 0
    for i, name in enumerate(("k", "v")):
        want = torch.cat([case.values(name, b, np.arange(c, c + m)) for b, (c, m) in enumerate(zip(case.ctx, case.counts))])
        assert torch.equal(out[:, 2 * i:2 * i + 2].double(), want)
