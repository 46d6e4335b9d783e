"""moe_cache8_append and moe_cache8_read: codes and scales exactly as defined (a power of two rounds nothing)."""
import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from cache8_helpers import Cache8, code_values
from round_ops_helpers import DEV, DT, i32, stream, word

pytestmark = pytest.mark.gpu


def rows_of(case, dtype="bf16", seed=1, spread=1.5, pad=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = int(case.start[-1])
    x = torch.randn((n, 2 * case.hkv, case.d + pad), generator=gen, device=DEV)
    x = (x * torch.exp2(spread * torch.randn((n, 2 * case.hkv, 1), generator=gen, device=DEV))).to(DT[dtype][0])
    if pad:
        x = x.reshape(n, -1)[:, :2 * case.hkv * case.d].unflatten(1, (2 * case.hkv, case.d))
    return {"k": x[:, :case.hkv], "v": x[:, case.hkv:]}


def append(case, rows, **kw):
    status = word()
    mv.moe_cache8_append(case.rows_args(rows["k"], rows["v"], status, **kw), stream())
    return int(status.item())


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,hkv", [(64, 1), (64, 8), (128, 3), (256, 2)])
def test_types_and_heads(fmt, dtype, d, hkv):
    case = Cache8(d + hkv, [0, 5, 30, 16], [3, 20, 1, 0], hkv=hkv, d=d, page=16, block=8, fmt=fmt)
    rows = rows_of(case, dtype)
    want = case.appended(rows)
    assert append(case, rows) == 0
    case.same(want)


@pytest.mark.parametrize("page,block", [(1, 1), (3, 1), (16, 16), (16, 1), (24, 8), (64, 4), (64, 64), (128, 128), (256, 32)])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_pages_blocks_and_layouts(page, block, layout, fmt):
    case = Cache8(page, [0, 1, 77, 130, 255], [1, 150, 7, 64, 3], hkv=2, d=64, page=page, block=block, fmt=fmt, layout=layout)
    rows = rows_of(case)
    want = case.appended(rows)
    assert append(case, rows) == 0
    case.same(want)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_a_block_filled_row_by_row(fmt):
    """Its scale goes up and down with what it holds; after each row codes and scale are as defined."""
    case = Cache8(3, [0], [1], hkv=2, d=64, page=32, block=16, fmt=fmt)
    case.table = np.array([[1, 0]])
    case.width = 2
    for i in range(40):
        case.ctx, case.start = [i], np.array([0, 1])
        rows = rows_of(case, seed=i, spread=4)
        want = case.appended(rows)
        assert append(case, rows) == 0
        case.same(want)


@pytest.mark.parametrize("scales", ["pow2", "any"])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_what_is_held_under_scales_of_any_value(fmt, scales):
    case = Cache8(4, [7, 20, 45], [2, 30, 4], hkv=3, d=128, page=16, block=16, fmt=fmt, scales=scales)
    rows = rows_of(case)
    want = case.appended(rows)
    assert append(case, rows) == 0
    case.same(want)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_borders_of_codes_and_scales(fmt):
    """Ties between codes, values at the largest code and just above it, zeros, the smallest and largest numbers."""
    case = Cache8(5, [0], [64], hkv=1, d=64, page=64, block=1, fmt=fmt)
    values = np.sort(code_values(fmt)[np.isfinite(code_values(fmt))])
    ties = (values[1:] + values[:-1]) / 2
    x = np.zeros((64, 64), np.float32)
    flat = np.concatenate([values, ties, np.nextafter(ties.astype(np.float32), np.float32(np.inf))]).astype(np.float32)
    x[:flat.size // 63 + 1, 1:] = np.resize(flat, (flat.size // 63 + 1, 63))
    x[:flat.size // 63 + 1, 0] = case.top  # the scale stays 1
    more = np.float32([case.top, np.nextafter(np.float32(case.top), np.float32(1e9)), 0, 1e-45, 1e-38, 3.4e38, -3.4e38, 2.0**-126, 2.0**-120, case.top * 2.0**-126])
    x[40:50, 0] = more
    x[40:50, 1] = -more / 3
    rows = {"k": torch.from_numpy(x).to(DEV)[:, None].contiguous(), "v": torch.from_numpy(x[::-1].copy()).to(DEV)[:, None].contiguous()}
    want = case.appended(rows)
    assert append(case, rows) == 0
    case.same(want)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_values_that_are_not_finite(fmt):
    case = Cache8(6, [5, 0], [6, 3], hkv=2, d=64, page=16, block=8, fmt=fmt)
    rows = rows_of(case)
    rows["k"][2, 0, 5] = float("inf")
    rows["k"][2, 1, 7] = float("nan")
    rows["v"][8, 1, 63] = -float("inf")
    want = case.appended(rows)
    assert append(case, rows) == mv.MOE_DEV_VALUE
    case.same(want)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -1.0, 1e-40])
def test_scales_that_are_none_count_as_zero(value):
    case = Cache8(7, [5], [2], hkv=2, d=64, page=16, block=16, fmt="e4m3")
    case.k_scale[int(case.table[0, 0]), 0, 1] = value
    rows = rows_of(case)
    want = case.appended(rows)
    assert append(case, rows) == mv.MOE_DEV_VALUE
    case.same(want)


def test_what_lies_behind_the_context_has_no_influence():
    """Rejected drafts in the same block: other bits there, the same block afterwards."""
    results = []
    for seed in (1, 2):
        case = Cache8(8, [11], [2], hkv=2, d=64, page=16, block=16, fmt="i8")
        page = int(case.table[0, 0])
        case.raw("k")[page, 11:] = torch.randint(0, 256, case.raw("k")[page, 11:].shape, dtype=torch.uint8,
                                                 generator=torch.Generator().manual_seed(seed)).to(DEV)
        rows = rows_of(case)
        assert append(case, rows) == 0
        results.append((case.raw("k")[page, :13].clone(), case.k_scale[page].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_rows_of_any_stride_many_requests_and_rows_of_nobody():
    rng = np.random.default_rng(9)
    ctx, n = rng.integers(0, 60, 700), rng.integers(0, 5, 700)
    case = Cache8(9, ctx.tolist(), n.tolist(), hkv=2, d=64, page=8, block=4, fmt="e4m3")
    rows = rows_of(case, pad=8)
    assert rows["k"].stride(0) == 2 * 2 * 72
    more = {m: torch.cat([rows[m], rows[m][:5] + 1]) for m in rows}  # five rows behind the last request's
    want = case.appended(rows)
    assert append(case, rows) == 0
    case.same(want)
    assert append(case, more) == 0  # again, and nothing of the rows of nobody
    case.same(case.appended(rows))


def test_bad_lengths_and_pages():
    ctx, n = [5, 9, 0, 40], [3, 4, 6, 2]
    case = Cache8(10, ctx, n, hkv=2, d=64, page=16, block=8, fmt="i8")
    rows = rows_of(case)
    want = case.appended(rows, only=[0, 2, 3])
    assert append(case, rows, ctx=i32([5, -1, 0, 40])) == mv.MOE_DEV_LENGTH
    case.same(want)
    want = case.appended(rows, only=[0, 1, 2])
    assert append(case, rows, ctx=i32([5, 9, 0, case.width * 16])) == mv.MOE_DEV_LENGTH
    case.same(want)
    case.table[2, 0] = case.n_pages
    table = case.table.copy()
    want = case.appended(rows)
    assert append(case, rows, table=i32(table)) == mv.MOE_DEV_INDEX
    case.same(want)
    # row starts that do not ascend: nothing outside the buffers is touched
    status = append(case, rows, start=i32([0, 9, 4, 2**31 - 1, 15]))
    assert status & mv.MOE_DEV_LENGTH


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,hkv,page,block,layout", [(64, 3, 24, 8, "hnd"), (128, 4, 16, 16, "nhd"), (256, 1, 3, 1, "nhd")])
def test_read(fmt, dtype, d, hkv, page, block, layout):
    case = Cache8(d, [0, 17, 3], [130, 40, 0], hkv=hkv, d=d, page=page, block=block, fmt=fmt, layout=layout, scales="any")
    n = int(case.start[-1])
    out = torch.full((n + 4, 2 * hkv, d), 7.0, dtype=DT[dtype][0], device=DEV)
    status = word()
    mv.moe_cache8_read(case.rows_args(out[:, :hkv], out[:, hkv:], status), stream())
    assert int(status.item()) == 0
    for i, name in enumerate(("k", "v")):
        want = torch.cat([case.values(name, b, np.arange(c, c + m)) for b, (c, m) in enumerate(zip(case.ctx, case.counts))])
        assert torch.equal(out[:n, i * hkv:(i + 1) * hkv], want.float().to(DT[dtype][0]))
    assert (out[n:] == 7).all()  # rows behind the last request's


def test_read_of_missing_pages_bad_scales_and_nan():
    case = Cache8(12, [0], [40], hkv=1, d=64, page=16, block=8, fmt="e4m3")
    case.k_scale[int(case.table[0, 0]), 0, 0] = float("nan")
    case.raw("v")[int(case.table[0, 2]), 3, 0, 5] = 0x7f
    case.table[0, 1] = -1
    out = torch.zeros((40, 2, 64), dtype=torch.float32, device=DEV)
    status = word()
    mv.moe_cache8_read(case.rows_args(out[:, :1], out[:, 1:], status), stream())
    assert int(status.item()) == mv.MOE_DEV_INDEX | mv.MOE_DEV_VALUE
    assert (out[16:32] == 0).all() and (out[:8, 0] == 0).all() and (out[8:16, 0] != 0).any()
    assert torch.isnan(out[35, 1, 5]) and int(torch.isnan(out).sum()) == 1


def test_append_then_read_gives_rows_within_half_a_step():
    """A value is off by half a step of its code at most: e4m3 2^-4 of it (2^-10 steps of the scale below the
    smallest normal code), int8 half a scale."""
    for fmt in ("e4m3", "i8"):
        case = Cache8(13, [0, 3], [50, 33], hkv=2, d=128, page=32, block=16, fmt=fmt)
        case.ctx = [0, 0]  # nothing held
        rows = rows_of(case)
        assert append(case, rows) == 0
        out = torch.empty((83, 4, 128), dtype=torch.float32, device=DEV)
        status = word()
        mv.moe_cache8_read(case.rows_args(out[:, :2], out[:, 2:], status), stream())
        assert int(status.item()) == 0
        r = 0
        for b, n in enumerate(case.counts):
            p, o = case.where(b, np.arange(n))
            for i, name in enumerate(("k", "v")):
                s = getattr(case, name + "_scale")[p, o // 16].double()[..., None]
                x = rows[name][r:r + n].double()
                step = torch.maximum(x.abs() * 2**-4, s * 2**-10) if fmt == "e4m3" else s / 2
                assert ((out[r:r + n, 2 * i:2 * i + 2].double() - x).abs() <= step).all()
            r += n


def test_another_stream_and_a_replayed_graph():
    case = Cache8(14, [10, 0], [4, 9], hkv=2, d=64, page=16, block=8, fmt="e4m3")
    rows = rows_of(case)
    rows = {m: x.contiguous() for m, x in rows.items()}
    status = word()
    args = case.rows_args(rows["k"], rows["v"], status)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        mv.moe_cache8_append(args, stream())
    for seed in (3, 4):
        fresh = rows_of(case, seed=seed)
        for m in rows:
            rows[m].copy_(fresh[m])
        torch.cuda.synchronize()
        want = case.appended(rows)
        graph.replay()
        torch.cuda.synchronize()
        case.same(want)
    assert int(status.item()) == 0


def test_a_cache_whose_offsets_pass_32_bits():
    case = Cache8(15, [16], [20], hkv=1, d=256, page=16, block=16, fmt="i8", spare=1)
    stride = 1 << 31
    view = torch.zeros(2 * stride + 4096, dtype=torch.int8, device=DEV).as_strided((3, 16, 1, 256), (stride, 256, 256, 1))
    case.n_pages, case.table, case.width = 3, np.array([[0, 2, 1]]), 3
    case.k = case.v = view  # (the same rows into both, blocks that hold nothing before)
    case.k_scale, case.v_scale = (torch.full((3, 1, 1), 0.5, device=DEV) for _ in range(2))
    x = torch.randn((20, 1, 256), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    want = case.appended({"k": x, "v": x})
    assert append(case, {"k": x, "v": x}) == 0
    case.same(want)
    out = torch.empty((20, 2, 256), dtype=torch.float32, device=DEV)
    status = word()
    mv.moe_cache8_read(case.rows_args(out[:, :1], out[:, 1:], status), stream())
    assert int(status.item()) == 0
    assert torch.equal(out[:, 0].double(), case.values("k", 0, np.arange(16, 36))[:, 0])


@pytest.mark.parametrize("moves", [False, True])
@pytest.mark.parametrize("d,block", [(64, 4), (64, 16), (256, 64)])
def test_held_nan_codes_become_zero_whether_the_scale_moves_or_not(d, block, moves):
    case = Cache8(16, [block + block // 2 + 1, 0], [1, 2], hkv=2, d=d, page=64, block=block, fmt="e4m3")
    p, o = (int(x) for x in case.where(0, np.array([block])))  # the first held position of the block
    for name in ("k", "v"):
        codes = case.raw(name)
        getattr(case, name + "_scale")[p, o // block] = 0.25
        codes[p, o, :, 0] = 0x7e  # the largest code: the scale stays where the rows are small
        codes[p, o + 1, 0, 3], codes[p, o + 1, 1, d - 1] = 0x7f, 0xff
    rows = {m: x * (1000 if moves else 0.01) for m, x in rows_of(case).items()}
    want = case.appended(rows)
    assert append(case, rows) == mv.MOE_DEV_VALUE
    case.same(want)
    held = case.raw("v")[p, o:o + block // 2 + 2].cpu().numpy()
    assert not np.isnan(code_values("e4m3")[held]).any()
    assert (float(case.v_scale[p, o // block, 0]) == 0.25) != moves


def appended_in_turn(fmt, block, steps, seed):
    """Appends of which some rows are rejected: (rows brought, rows that stay, their size) a step.  Returns the case, the rows
    that stayed in 64 bits, and for each the largest scale that its block had from then on."""
    total = sum(keep for _, keep, _ in steps) + max(n for n, _, _ in steps)
    case = Cache8(seed, [0], [total], hkv=2, d=64, page=64, block=block, fmt=fmt)
    ctx, kept, largest = 0, np.zeros((total, 2, 64)), np.zeros((total, 2))
    for i, (n, keep, size) in enumerate(steps):
        case.ctx, case.counts, case.start = [ctx], [n], np.array([0, n])
        rows = {m: x * size for m, x in rows_of(case, "f32", seed=i, spread=0.3).items()}
        want = case.appended(rows)
        assert append(case, rows) == 0
        case.same(want)
        kept[ctx:ctx + keep] = rows["v"][:keep].double().cpu().numpy()
        p, o = case.where(0, np.arange(total))
        scale = case.v_scale[p, o // block].double().cpu().numpy()
        largest[ctx:ctx + keep] = 0
        for at in range(ctx // block * block, ctx + keep):
            largest[at] = np.maximum(largest[at], scale[at])
        ctx += keep
    return case, kept[:ctx], largest[:ctx]


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("block", [1, 8, 64])
def test_what_rejected_rows_leave_of_the_rows_before_them(fmt, block):
    """A held value was rounded at every larger scale that its block has had, that of rows which were rejected since
    included: off by less than one step of the largest (int8), or of its smallest codes beside the first rounding (e4m3)."""
    rng = np.random.default_rng(block)
    steps = []
    for _ in range(40):
        n = int(rng.integers(1, 7))
        steps.append((n, int(rng.integers(1, n + 1)), float(2.0 ** rng.integers(-6, 8))))
    case, kept, largest = appended_in_turn(fmt, block, steps, 17)
    got = case.values("v", 0, np.arange(len(kept))).cpu().numpy()
    bound = largest[..., None] if fmt == "i8" else np.abs(kept) * 2.0**-4 + largest[..., None] * 2.0**-9
    assert (np.abs(got - kept) < bound).all()


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_a_large_row_that_was_rejected_leaves_its_rounding_unless_it_had_a_block_of_its_own(fmt):
    """Rows of about 1, a row 2^12 times as large, rejected, a row of about 1: the scale is small again, and the first
    rows are as the large scale left them; behind the end of a block they are as they were written."""
    far = {}
    for held in (5, 8):
        case, kept, largest = appended_in_turn(fmt, 8, [(held, held, 1.0), (1, 0, 4096.0), (1, 1, 1.0)], 18)
        got = case.values("v", 0, np.arange(held)).cpu().numpy()
        p, o = case.where(0, np.arange(held))
        step = case.v_scale[p, o // 8].double().cpu().numpy()[..., None] * (1 if fmt == "i8" else 2.0**-9)
        off = np.abs(got - kept[:held]) - (0 if fmt == "i8" else np.abs(kept[:held]) * 2.0**-4)
        far[held] = float((off / step).max())
        large = largest[:held, :, None] * (1 if fmt == "i8" else 2.0**-9)
        assert (off < large).all()
    assert far[8] <= 0.5 and far[5] > 8


@pytest.mark.parametrize("first", [-2**31, -2**31 + 5, -2**31 + 40, -2**30, -1])
def test_row_starts_as_far_below_zero_as_they_go(first):
    """The request that begins there, and the one that ends there, are left out; the others are worked on as ever."""
    ctx, n = [5, 9, 0, 40], [3, 4, 6, 2]
    case = Cache8(24, ctx, n, hkv=2, d=64, page=16, block=8, fmt="e4m3")
    rows = rows_of(case)
    start = i32([0, first, 7, 13, 15])
    want = case.appended(rows, only=[2, 3])
    assert append(case, rows, start=start) == mv.MOE_DEV_LENGTH
    case.same(want)
    out = torch.full((15, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    status = word()
    mv.moe_cache8_read(case.rows_args(out[:, :2], out[:, 2:], status, start=start), stream())
    assert int(status.item()) == mv.MOE_DEV_LENGTH
    for i, name in enumerate(("k", "v")):
        want = torch.cat([case.values(name, b, np.arange(ctx[b], ctx[b] + n[b])) for b in (2, 3)])
        assert torch.equal(out[7:, 2 * i:2 * i + 2], want.float().bfloat16())
    assert (out[:7] == 7).all()


@pytest.mark.parametrize("hkv", [8, 32])
def test_thread_blocks_beside_each_other_share_the_same_tasks(hkv):
    """Few rows, many blocks that begin among them: each of the thread blocks that share them takes its part of one
    order, every time."""
    case = Cache8(19, [0, 3, 1], [16, 7, 9], hkv=hkv, d=256, page=4, block=1, fmt="i8")
    for seed in range(10):
        rows = rows_of(case, seed=seed)
        want = case.appended(rows)
        assert append(case, rows) == 0
        case.same(want)
