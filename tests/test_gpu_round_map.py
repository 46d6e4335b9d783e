"""moe_round_map against a plain request-by-request build of the same map: whole numbers, so equality."""
import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from round_ops_helpers import DEV, MapCase, at, i32, word
from spec_verify_layer_gb300 import MOE_DEV_INDEX, MOE_DEV_LENGTH, MOE_DEV_PAGES

pytestmark = pytest.mark.gpu


def same(case, **kw):
    got, status = case.run(**kw)
    want = case.plain(**{k: v for k, v in kw.items() if k in ("free", "rows")})
    for name, w in want.items():
        if got[name] is not None:
            np.testing.assert_array_equal(got[name], w, err_msg=name)
    return got, status


@pytest.mark.parametrize("page", [1, 3, 16, 64, 256])
@pytest.mark.parametrize("req", [1, 5, 255, 256, 257, 600])
@pytest.mark.parametrize("tree", [False, True])
def test_map(req, page, tree):
    rng = np.random.default_rng(req * page + tree)
    ctx, new = rng.integers(0, 300, req), rng.integers(0, 65 if tree else 40, req)
    ctx[rng.random(req) < 0.2] = 0
    new[rng.random(req) < 0.2] = 0
    for held, extra in ((True, 2), (True, 0), (False, 0)):
        case = MapCase(req, ctx, new, page, extra=extra, tree=tree, held=held, pad=int(rng.integers(0, 9)))
        _, status = same(case, mask=tree)
        assert status == 0


@pytest.mark.parametrize("new", [[0], [0, 0, 0], [1], [64], [63, 64, 1]])
def test_small_and_full_trees_and_chains(new):
    for tree in (False, True):
        _, status = same(MapCase(1, [7] * len(new), new, 16, tree=tree))
        assert status == 0


def test_a_chain_as_the_deepest_tree():
    case = MapCase(2, [5, 100], [64, 64], 16, tree=True)
    case.parents = np.array(list(range(-1, 63)) * 2)
    same(case)


def test_prompts_over_many_blocks():
    rng = np.random.default_rng(0)
    case = MapCase(3, rng.integers(0, 3000, 700), rng.integers(0, 900, 700), 16, pad=3)
    _, status = same(case, mask=False)
    assert status == 0


def test_trees_across_block_borders():
    """Rows of one tree on both sides of a block's step of rows."""
    case = MapCase(4, [9] * 130, [61] * 130, 8, tree=True)
    same(case)


def test_free_pages_run_out():
    case = MapCase(5, [10, 20, 30], [40, 50, 60], 8, spare=0)
    got, status = same(case, free=case.free[:7])
    assert status == MOE_DEV_PAGES and (got["row_slot"] == -1).any()
    got, status = same(case, free=case.free[:0])
    assert status == MOE_DEV_PAGES and got["taken"][0] == 0


def test_table_columns_run_out():
    case = MapCase(6, [10, 0, 3], [40, 3, 100], 8, width=4)
    got, status = case.run(mask=False)
    want = case.plain()
    assert status == MOE_DEV_PAGES
    for name in ("table", "pages", "row_slot", "row_pos", "row_start"):
        np.testing.assert_array_equal(got[name], want[name], err_msg=name)


def test_more_rows_than_the_arrays_hold():
    case = MapCase(7, [3, 4, 5], [10, 10, 10], 4)
    got, status = same(case, rows=17, mask=False)
    assert status == MOE_DEV_LENGTH and got["row_start"][-1] == 17


def test_no_rows_at_all():
    got, status = same(MapCase(8, [3, 0], [0, 0], 4))
    assert status == 0 and got["row_start"][-1] == 0


def test_lengths_that_make_no_sense():
    case = MapCase(9, [5, 3, 7, 8], [4, 6, 100, 2], 16, held=False, width=8)
    case.ctx = np.array([5, -3, 2**31 - 5, 8])
    # the second and third request bring nothing; the held pages of the third do not fit the table
    got, status = case.run(rows=10)
    assert status & MOE_DEV_LENGTH
    np.testing.assert_array_equal(got["row_start"], [0, 4, 4, 4, 6])
    np.testing.assert_array_equal(got["row_req"], [0] * 4 + [3] * 2 + [-1] * 4)


def test_held_pages_that_do_not_cover_the_context():
    case = MapCase(10, [40], [4], 16)
    case.held = np.array([1])
    got, status = case.run()
    assert status == MOE_DEV_LENGTH and got["row_req"].tolist() == [0] * 4


def test_parents_out_of_range_count_as_none():
    case = MapCase(11, [6], [6], 16, tree=True)
    case.parents = np.array([-1, 0, 2, -2, 7, 3])
    got, status = case.run()
    assert status == MOE_DEV_INDEX
    assert got["mask"].tolist() == [1, 3, 4, 8, 16, 40]
    assert got["row_pos"].tolist() == [6, 7, 6, 6, 6, 7]


def test_pages_outside_the_pool():
    case = MapCase(12, [5, 9], [20, 7], 8)
    bad = case.free.copy()
    bad[0], bad[1] = -4, 10**6
    got, status = case.run(free=bad)
    assert status == MOE_DEV_INDEX
    pages = got["row_slot"] // 8
    assert ((pages >= -1) & (pages < case.n_pages)).all() and (got["row_slot"] == -1).any()


def test_trees_of_more_than_64_rows_are_reported():
    case = MapCase(13, [0], [70], 16)
    case.parents = np.arange(-1, 69)
    got, status = case.run()
    assert status == MOE_DEV_LENGTH
    assert (got["mask"][64:] == 0).all() and got["mask"][63] == -1


def test_a_captured_map_follows_its_lengths():
    import spec_verify_layer_gb300 as mv
    from round_ops_helpers import DEV, at, i32, word
    side = torch.cuda.Stream()
    a, b = MapCase(14, [5, 40, 17], [3, 9, 0], 8), MapCase(15, [30, 1, 0], [12, 2, 7], 8)
    width, rows, pool = 12, 24, 64
    ctx, new, free = i32([0] * 3), i32([0] * 3), i32(range(40, 40 + 12))
    table = i32(np.arange(36).reshape(3, 12) % 40)
    outs = [i32([0] * n) for n in (4, 3, 1, rows, rows, rows)]
    status = word()
    args = mv.make_map_args(n_req=3, n_rows=rows, page_size=8, n_pages=pool, table_width=width, n_free=12,
                            ctx_len=at(ctx), new_len=at(new), free_pages=at(free), block_table=at(table),
                            row_start=at(outs[0]), pages=at(outs[1]), n_taken=at(outs[2]), row_req=at(outs[3]),
                            row_pos=at(outs[4]), row_slot=at(outs[5]), dev_status=at(status))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mv.moe_round_map(args, torch.cuda.current_stream().cuda_stream)
    for case in (a, b, a):
        case.width, case.table, case.free, case.held = width, np.arange(36).reshape(3, 12) % 40, np.arange(40, 52), (
            -(-case.ctx // 8))
        want = case.plain(rows=rows)
        table.copy_(i32(case.table))
        ctx.copy_(i32(case.ctx))
        new.copy_(i32(case.new))
        graph.replay()
        torch.cuda.synchronize()
        for t, name in zip([table] + outs, ("table", "row_start", "pages", "taken", "row_req", "row_pos", "row_slot")):
            np.testing.assert_array_equal(t.cpu().numpy(), want[name], err_msg=name)
    assert int(status.item()) == 0 and DEV == "cuda"


class Map:
    """A case's tensors and its descriptor, for calls that are made more than once."""

    def __init__(self, case, in_place=False):
        self.ctx, self.new, self.held, self.table = (i32(getattr(case, n)) for n in ("ctx", "new", "held", "table"))
        self.free, self.status, B, rows = i32(case.free), word(), len(case.ctx), case.rows
        self.parents = None if case.parents is None else i32(case.parents)
        self.row_start, self.taken = i32([-7] * (B + 1)), i32([-7])
        self.pages = self.held if in_place else i32([-7] * B)
        self.row_req, self.row_pos, self.row_slot = (i32([-7] * rows) for _ in range(3))
        self.mask = torch.zeros(rows, dtype=torch.int64, device=DEV)
        self.args = mv.make_map_args(
            n_req=B, n_rows=rows, page_size=case.page, n_pages=case.n_pages, table_width=case.width,
            n_free=self.free.numel(), ctx_len=at(self.ctx), new_len=at(self.new), pages_held=at(self.held),
            free_pages=at(self.free), parents=at(self.parents), block_table=at(self.table),
            row_start=at(self.row_start), pages=at(self.pages), n_taken=at(self.taken), row_req=at(self.row_req),
            row_pos=at(self.row_pos), row_slot=at(self.row_slot), tree_mask=at(self.mask) if self.parents is not None else 0,
            dev_status=at(self.status))

    def call(self, side=None):
        mv.moe_round_map(self.args, (side or torch.cuda.current_stream()).cuda_stream)

    def got(self):
        names = ("table", "row_start", "pages", "taken", "row_req", "row_pos", "row_slot", "mask")
        return {n: getattr(self, n).cpu().numpy().astype(np.int64) for n in names}


@pytest.mark.parametrize("req,new,page,tree", [(6, 16, 16, True), (700, 900, 16, False), (130, 61, 8, True),
                                               (5200, 3, 16, False), (3, 0, 4, False)])
def test_held_pages_in_place(req, new, page, tree):
    """`pages` over `pages_held`: every block reads what was held, whichever has ended."""
    rng = np.random.default_rng(req)
    case = MapCase(18, rng.integers(0, 300, req), rng.integers(0, new + 1, req), page, extra=2, tree=tree, pad=3)
    t = Map(case, in_place=True)
    t.call()
    got, want = t.got(), case.plain()
    for name in got:
        if name != "mask" or tree:
            np.testing.assert_array_equal(got[name], want[name], err_msg=name)
    assert int(t.status.item()) == 0


def test_rounds_in_place_in_a_graph():
    """Round after round of one captured call: what a round leaves in the held pages is the next one's input."""
    case = MapCase(19, [0] * 40, [37] * 40, 8, spare=2000, width=64)
    t = Map(case, in_place=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mv.moe_round_map(t.args, torch.cuda.current_stream().cuda_stream)
    for _ in range(6):
        want = case.plain()
        t.free.copy_(i32(np.resize(case.free, t.free.numel())))
        graph.replay()
        torch.cuda.synchronize()
        got = t.got()
        for name in got:
            if name != "mask":
                np.testing.assert_array_equal(got[name], want[name], err_msg=name)
        case.ctx, case.held, case.table = case.ctx + case.new, want["pages"], want["table"]
        case.free = case.free[int(want["taken"][0]):]
        t.ctx.copy_(i32(case.ctx))
    assert int(t.status.item()) == 0


def test_counts_of_pages_in_place_when_free_pages_run_out():
    case = MapCase(20, [10, 20, 30], [40, 50, 60], 8, spare=0)
    case.free = case.free[:7]
    t = Map(case, in_place=True)
    t.call()
    want = case.plain()
    assert int(t.status.item()) == MOE_DEV_PAGES
    np.testing.assert_array_equal(t.got()["pages"], want["pages"])
    np.testing.assert_array_equal(t.got()["table"], want["table"])


def test_calls_of_different_sizes_from_two_threads():
    """Calls with many requests, which take more shared memory than the default, of different counts side by side."""
    import threading
    cases = [MapCase(16, [5] * 16384, [0] * 16383 + [3], 16), MapCase(17, [5] * 5200, [0] * 5199 + [3], 16)]
    errors, go = [], threading.Barrier(2)

    def work(case):
        try:
            t = Map(case)
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            go.wait()
            for _ in range(3000):
                t.call(side)
            side.synchronize()
            assert int(t.status.item()) == 0
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
