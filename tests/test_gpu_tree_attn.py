"""moe_tree_attention against softmax attention in 64 bits; the bound of each element is derived in TreeCase.check.

Every cache slot that holds no position is NaN, so a read past a length shows.
"""
import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from round_ops_helpers import DEV, TreeCase, at, i32, stream, word

pytestmark = pytest.mark.gpu


def good(case, **kw):
    out, lse, status = case.run(**kw)
    assert status == 0
    case.check(out, lse)
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (6, 2), (16, 1), (24, 8), (32, 4)])
def test_heads_and_types(dtype, d, hq, hkv):
    good(TreeCase(d + hq, [0, 5, 130, 64, 63], [3, 1, 9, 0, 1], hq=hq, hkv=hkv, d=d, page=16, dtype=dtype))


@pytest.mark.parametrize("n", [1, 2, 7, 15, 16, 17, 33, 63, 64])
@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
def test_tree_widths_and_masks(n, mask):
    good(TreeCase(n, [0, 200, 61], [n, n, max(0, n - 1)], hq=8, hkv=2, d=128, page=16, dtype="bf16", mask=mask))


@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 256])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_pages_and_layouts(page, layout):
    good(TreeCase(page, [77, 300, 0, 255], [4, 6, 5, 1], hq=6, hkv=3, d=64, page=page, dtype="f16", layout=layout))


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1000, 4097])
def test_context_lengths(ctx):
    good(TreeCase(ctx, [ctx], [5], hq=8, hkv=1, d=128, page=16, dtype="bf16"))
    good(TreeCase(ctx, [ctx], [1], hq=4, hkv=4, d=64, page=16, dtype="f16"))


@pytest.mark.parametrize("hq,hkv,n", [(32, 4, 16), (32, 4, 64), (8, 8, 1), (16, 1, 64), (64, 1, 40), (128, 2, 3)])
def test_long_contexts_split_over_blocks(hq, hkv, n):
    good(TreeCase(hq + n, [20011], [n], hq=hq, hkv=hkv, d=128, page=64, dtype="bf16"))


def test_ragged_batches():
    rng = np.random.default_rng(0)
    for seed, req in ((1, 70), (2, 300)):
        ctx = rng.integers(0, 700, req)
        ctx[::7] = 0
        n = rng.integers(0, 20, req)
        good(TreeCase(seed, ctx.tolist(), n.tolist(), hq=8, hkv=2, d=64, page=16, dtype="bf16"))


@pytest.mark.parametrize("req", [383, 384, 385, 900])
def test_more_requests_than_threads(req):
    rng = np.random.default_rng(req)
    ctx = rng.integers(0, 200, req)
    n = rng.integers(0, 5, req)
    n[::11] = 0
    good(TreeCase(req, ctx.tolist(), n.tolist(), hq=4, hkv=1, d=64, page=16, dtype="bf16"))


def test_many_groups_of_query_rows():
    """Sixty-four heads to a key and 64 rows: sixteen groups of 256 query rows, some requests with fewer."""
    good(TreeCase(19, [700, 40, 0], [64, 9, 33], hq=64, hkv=1, d=128, page=16, dtype="bf16"))
    good(TreeCase(20, [300, 1], [20, 3], hq=128, hkv=2, d=64, page=16, dtype="f16"))
    good(TreeCase(21, [3000], [24], hq=64, hkv=1, d=256, page=32, dtype="bf16"))


@pytest.mark.parametrize("d", [64, 256])
def test_long_contexts_of_other_head_sizes(d):
    good(TreeCase(22, [15000, 8000], [16, 33], hq=16, hkv=2, d=d, page=24, dtype="f16", layout="hnd"))


def test_one_long_request_among_short_ones():
    good(TreeCase(3, [3, 9000, 0, 17, 40], [2, 20, 1, 0, 64], hq=16, hkv=2, d=128, page=32, dtype="bf16"))


def test_empty_rows():
    """No context and an empty mask: zeros and -infinity, whatever the tree's own values are."""
    case = TreeCase(4, [0, 0, 40], [6, 1, 3], hq=4, hkv=2, d=64, page=16, dtype="bf16", mask="random")
    case.mask[0] = 0
    case.mask[6] = 0
    out, lse = good(case)
    assert (out[0] == 0).all() and (lse[6] == -float("inf")).all()


def test_all_requests_empty():
    case = TreeCase(5, [10, 0], [0, 0], hq=4, hkv=2, d=64, page=16, dtype="bf16")
    case.run()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n,hq", [(5, 4), (16, 32), (64, 16)])
def test_masked_infinities_and_nan_have_no_influence(value, n, hq):
    """A tree row whose cached key and value are not finite changes only the rows that see it."""
    case = TreeCase(6, [90], [n], hq=hq, hkv=2, d=128, page=16, dtype="bf16")
    clean, clean_lse = good(case)
    seen = case.seen(0)[:, 90:]
    j = n // 2
    p, o = case.where(0, np.array([90 + j]))
    for cache in (case.k, case.v):
        cache[p, o] = value
    out, lse, status = case.run()
    blind = ~seen[:, j]
    assert status == 0 and blind.any()
    assert torch.equal(out[blind], clean[blind]) and torch.equal(lse[blind], clean_lse[blind])
    assert not torch.isfinite(out[j].float()).any()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_seen_value_that_is_not_finite_shows_where_it_belongs(value):
    case = TreeCase(7, [40], [12], hq=8, hkv=2, d=64, page=16, dtype="f16")
    clean, _ = good(case)
    seen = case.seen(0)[:, 40:]
    p, o = case.where(0, np.array([43]))
    case.v[p, o, 1, 9] = value
    out, lse, _ = case.run()
    touched = torch.zeros((12, 8, 64), dtype=torch.bool, device=DEV)
    touched[seen[:, 3], 4:, 9] = True
    assert torch.equal(out[~touched], clean[~touched])
    assert not torch.isfinite(out[touched].float()).any()


def test_large_scores():
    """Scores of a few thousand: the maximum is taken out before the exponential."""
    good(TreeCase(8, [500, 3], [7, 2], hq=4, hkv=1, d=128, page=16, dtype="bf16", scale=10.0))
    good(TreeCase(9, [500, 3], [7, 2], hq=4, hkv=1, d=128, page=16, dtype="bf16", scale=-0.3))
    good(TreeCase(9, [500, 3], [7, 2], hq=4, hkv=1, d=128, page=16, dtype="bf16", scale=0.0))


def test_the_maximum_comes_last():
    """Scores that rise along the context: every tile moves the running maximum."""
    case = TreeCase(10, [3000], [4], hq=4, hkv=1, d=64, page=16, dtype="bf16")
    p, o = case.where(0, np.arange(3004))
    ramp = torch.linspace(0, 3, 3004, device=DEV)[:, None]
    case.q.fill_(0.5)
    case.k[p, o, 0] = ramp.expand(-1, 64).to(case.dt)
    good(case)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,n", [(64, 4), (64, 40), (128, 4), (128, 40), (256, 4), (256, 40)])
@pytest.mark.parametrize("levels", ["rise", "fall", "rise within tiles", "saw"])
def test_scores_in_steps(dtype, d, n, levels):
    """Scores that go up or down by far more than a weight's range, between tiles and inside them; rows of the
    same request see them with either sign, or not at all."""
    case = TreeCase(26, [900, 40], [n, 3], hq=4, hkv=1, d=d, page=16, dtype=dtype, q_scale=0.5)
    pos = torch.arange(900 + n, device=DEV)
    level = {"rise": 12 * (pos // 64), "fall": -12 * (pos // 64), "rise within tiles": 40 * (pos // 32 % 4),
             "saw": 60 * (pos // 64 % 2) + pos // 128}[levels].float()
    p, o = case.where(0, np.arange(900 + n))
    case.k[p, o, 0, 0] = level.to(case.dt)
    case.q[:, :, 0] = (torch.tensor([1.0, -1.0, 0.0, 1.0], device=DEV) * d ** 0.5).to(case.dt)
    good(case)


def test_strided_queries_and_padding_rows():
    case = TreeCase(11, [30, 100], [5, 8], hq=6, hkv=2, d=64, page=16, dtype="bf16", pad_rows=4, q_pad=128)
    out, lse, status = case.run()
    assert status == 0
    case.check(out, lse)
    assert torch.isnan(out[13:].float()).all() and torch.isnan(lse[13:]).all()  # not written


def test_without_lse_and_with_a_wider_bound():
    case = TreeCase(12, [30, 100], [5, 8], hq=8, hkv=2, d=128, page=16, dtype="bf16")
    out, lse = good(case)
    wide, wide_lse, status = case.run(max_tree=64)
    assert status == 0
    case.check(wide, wide_lse)
    o2, _ = case.outputs()
    status = word()
    args = case.args(o2, None, status)
    ws = torch.zeros(mv.moe_tree_attention_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    mv.moe_tree_attention(args, at(ws), ws.numel(), stream())
    assert torch.equal(o2, out)


def test_repeats_are_equal_bit_for_bit():
    case = TreeCase(13, [5000, 12, 700], [16, 3, 30], hq=16, hkv=2, d=128, page=16, dtype="bf16")
    out, lse, _ = case.run()
    for _ in range(3):
        o2, l2, status = case.run(times=3)
        assert status == 0 and torch.equal(out, o2) and torch.equal(lse, l2)


def test_rows_do_not_depend_on_what_ran_before():
    """Row counts that leave lanes of a warp without a row: whatever an earlier call left there has no say."""
    case = TreeCase(23, [2000, 300, 41], [5, 3, 7], hq=6, hkv=2, d=64, page=24, dtype="f16", layout="hnd")
    out, lse, _ = case.run()
    for seed in (24, 25):
        TreeCase(seed, [900, 80], [40, 64], hq=16, hkv=2, d=64, page=16, dtype="f16", q_scale=30.0).run()
        o2, l2, status = case.run()
        assert status == 0 and torch.equal(out, o2) and torch.equal(lse, l2)


def test_bad_lengths_are_reported_and_left_out():
    case = TreeCase(14, [30, 100, 20], [5, 8, 2], hq=8, hkv=2, d=64, page=16, dtype="bf16")
    out, lse, status = case.run(ctx=i32([30, 10**6, -4]))
    assert status == mv.MOE_DEV_LENGTH
    case.check(out, lse, only=[0])
    assert (out[5:] == 0).all() and (lse[5:] == -float("inf")).all()
    out, lse, status = case.run(max_tree=5)
    assert status == mv.MOE_DEV_LENGTH
    case.check(out, lse, only=[0, 2])
    assert (out[5:13] == 0).all()


def test_row_starts_that_do_not_ascend_are_reported():
    case = TreeCase(15, [30, 100, 20], [5, 8, 2], hq=8, hkv=2, d=64, page=16, dtype="bf16")
    for start in ([0, 5, 3, 15], [0, 5, 13, 99], [-3, 5, 13, 15]):
        _, _, status = case.run(start=i32(start))
        assert status & mv.MOE_DEV_LENGTH, start


def test_pages_outside_the_cache_count_as_unseen():
    case = TreeCase(16, [100, 40], [3, 2], hq=4, hkv=2, d=64, page=16, dtype="bf16")
    table = i32(case.table)
    table[0, 2], table[0, 4] = -1, case.n_pages
    out, lse, status = case.run(table=table)
    assert status == mv.MOE_DEV_INDEX
    case.check(out, lse, only=[1])
    hidden = torch.zeros((3, 103), dtype=torch.bool, device=DEV)
    hidden[:, 32:48] = hidden[:, 64:80] = True
    full = TreeCase.seen
    case.seen = lambda b: full(case, b) & ~hidden
    case.check(out, lse, only=[0])


def test_another_stream_and_a_captured_round():
    case = TreeCase(17, [900, 40], [16, 7], hq=16, hkv=2, d=128, page=16, dtype="bf16")
    want, want_lse = good(case)
    out, lse = case.outputs()
    status, ctx = word(), i32(case.ctx)
    args = case.args(out, lse, status, ctx=ctx)
    ws = torch.zeros(mv.moe_tree_attention_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mv.moe_tree_attention(args, at(ws), ws.numel(), side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mv.moe_tree_attention(args, at(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    short = TreeCase(17, [900, 40], [16, 7], hq=16, hkv=2, d=128, page=16, dtype="bf16")
    for lens in (case.ctx, [333, 40], [0, 0], case.ctx):
        # the same cache seen with other context lengths: the tree's rows move to the positions after them
        ctx.copy_(i32(lens))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        short.k, short.v, short.table, short.q, short.mask = case.k, case.v, case.table, case.q, case.mask
        short.ctx = list(lens)
        short.check(out, lse)
    assert int(status.item()) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


def test_offsets_past_32_bits():
    """Pages at the end of a cache of more than 2^32 elements."""
    case = TreeCase(18, [300, 70], [8, 3], hq=8, hkv=2, d=128, page=64, dtype="bf16")
    n_pages = 2**32 // (64 * 2 * 128) + 40
    k = torch.zeros(n_pages * 64 * 2 * 128, dtype=torch.bfloat16, device=DEV).view(n_pages, 64, 2, 128)
    v = torch.zeros_like(k)
    far = n_pages - case.n_pages
    k[far:], v[far:] = case.k, case.v
    case.k, case.v, case.n_pages = k, v, n_pages
    case.table = np.where(case.table >= 0, case.table + far, -1)
    good(case)


def test_waits_that_give_up_are_reported_and_the_next_call_is_whole():
    """A bound of 1 ns makes waits give up in every role of the kernel and between blocks: the call ends, says so, and
    leaves nothing behind but its workspace's counters."""
    cases = [TreeCase(29, [9000, 300, 17], [16, 40, 3], hq=16, hkv=2, d=d, page=24, dtype="bf16") for d in (64, 128, 256)]
    for case in cases:
        want, want_lse, status = case.run()
        assert status == 0
        try:
            mv.moe_set_attention_wait_limit_ns(1)
            for _ in range(3):
                _, _, status = case.run()
                assert status == mv.MOE_DEV_TIMEOUT
        finally:
            mv.moe_set_attention_wait_limit_ns(0)
        out, lse, status = case.run()
        assert status == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("d,n", [(64, 3), (128, 2), (128, 40), (256, 3)])
@pytest.mark.parametrize("strong", [0, 3000, 5999])
def test_a_flat_tail_beside_one_strong_key(d, n, strong):
    """Weights of 2^-25.6 beside one of 1 in fp16: six thousand of them are the whole result where the strong key's
    value is 0.  A weight may be off by 2^-32 of the largest beside the half step of its type."""
    case = TreeCase(27, [6000] * 20, [n] * 20, hq=2, hkv=2, d=d, page=64, dtype="f16")
    case.q.zero_()
    case.q[:, :, 0] = d ** 0.5
    case.k[:, :, :, 0] = 0
    case.v[torch.isfinite(case.v)] = 1.0
    for b in range(20):
        p, o = case.where(b, np.array([strong]))
        case.k[p, o, :, 0] = 17.75
        case.v[p, o] = 0
    out, lse, status = case.run()
    assert status == 0
    case.check(out, lse, weight_step=2**-32)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_small_weights_keep_their_bits(d):
    """Spread scores: most weights are far below the largest one."""
    case = TreeCase(28, [9000, 700, 0], [7, 33, 20], hq=4, hkv=1, d=d, page=24, dtype="f16", q_scale=4.0, layout="hnd")
    out, lse, status = case.run()
    assert status == 0
    case.check(out, lse, weight_step=2**-32)
