"""moe_verify_drafts against the definition walked row by row in 64 bits.

The outputs are whole numbers, equal unless a decision lies nearer to its border than the call's sums are exact; the
walk says how near (1e-6 relative is what the header promises), and no case's inputs come that near.
"""
import math

import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from round_ops_helpers import DEV, DT, at, i32, stream, word

pytestmark = pytest.mark.gpu


class VerifyCase:
    def __init__(self, seed, counts, vocab, *, dtype="f32", mode="lookup", tree=False, temp=1.0, masked=False, pad=0, odd=0,
                 draft_dtype=None):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.counts, self.vocab, self.mode, self.tree = list(counts), vocab, mode, tree
        self.dt, self.code = DT[dtype]
        self.qt, self.qcode = DT[draft_dtype or dtype]
        self.inv = math.inf if mode == "greedy" else float(np.float32(1 / temp))
        self.start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        n = self.rows = int(self.start[-1]) + pad
        x = torch.randn((n, vocab + odd), generator=gen, device=DEV) * 2
        peaks = torch.randint(0, vocab, (n, 5), generator=gen, device=DEV)
        x.scatter_add_(1, peaks, 5 + 3 * torch.rand((n, 5), generator=gen, device=DEV))
        if masked:
            x.masked_fill_(torch.rand((n, vocab + odd), generator=gen, device=DEV) < 0.4, -math.inf)
        self.x = x.to(self.dt)[:, :vocab]
        self.parents = np.full(n, -1)
        for b, m in enumerate(self.counts):
            for i in range(1, m):
                self.parents[self.start[b] + i] = int(rng.integers(max(-1, i - 4), i)) if tree else i - 1
        above = np.zeros(n, np.int64)
        for b, m in enumerate(self.counts):
            for i in range(m):
                above[self.start[b] + i] = self.start[b] + max(0, self.parents[self.start[b] + i])
        above = torch.from_numpy(above).to(DEV)
        self.q = None
        if mode == "drawn":
            logits = self.x[above].float() + torch.randn((n, vocab), generator=gen, device=DEV)
            self.q = torch.softmax(logits, -1).to(self.qt)
            race = torch.empty((n, vocab), device=DEV).exponential_(generator=gen)
            tokens = (self.q.float() / race).argmax(-1)
        else:
            tokens = peaks[above, torch.randint(0, 5, (n,), generator=gen, device=DEV)]
            tokens = torch.where(torch.rand(n, generator=gen, device=DEV) < 0.05, -1, tokens)
        self.tokens = tokens.cpu().numpy().astype(np.int64)
        self.u = torch.rand(n, generator=gen, device=DEV)
        self.noise = torch.empty((len(self.counts), vocab + odd), device=DEV).exponential_(generator=gen)[:, :vocab]

    def args(self, outs, status, **kw):
        greedy = self.mode == "greedy"
        self.keep = [i32(self.start), i32(self.parents), i32(self.tokens)]
        d = dict(n_req=len(self.counts), n_rows=self.rows, vocab=self.vocab, dtype=self.code, logits=at(self.x), stride=self.x.stride(0),
                 row_start=at(self.keep[0]), parents=at(self.keep[1]) if self.tree else 0, tokens=at(self.keep[2]),
                 uniform=0 if greedy else at(self.u), noise=0 if greedy else at(self.noise), noise_stride=self.noise.stride(0),
                 draft_probs=at(self.q), draft_dtype=self.qcode, draft_stride=self.vocab, inv_temperature=self.inv,
                 accepted=at(outs[0]), path=at(outs[1]), next_token=at(outs[2]), dev_status=at(status))
        d.update(kw)
        return mv.make_verify_args(**d)

    def outputs(self):
        return i32([-9] * len(self.counts)), i32([-9] * max(1, self.rows)), i32([-9] * len(self.counts))

    def run(self, times=1, **kw):
        outs, status = self.outputs(), word()
        args = self.args(outs, status, **kw)
        ws = torch.zeros(mv.moe_verify_drafts_workspace_bytes(args), dtype=torch.uint8, device=DEV)
        assert ws.numel() > 0
        for _ in range(times):
            mv.moe_verify_drafts(args, at(ws), ws.numel(), stream())
        return [t.cpu().numpy().astype(np.int64) for t in outs], int(status.item())

    def probs(self, r):
        z = self.x[r].double() * self.inv
        if not (z > -math.inf).any():
            return torch.zeros_like(z)
        return torch.softmax(z, -1)

    def plain(self, near=2e-6):
        """Row after row by the definition; asserts that no decision is within `near` of its border."""
        accepted, path, follow = [], np.full(max(1, self.rows), -9), []
        for b, n in enumerate(self.counts):
            s = int(self.start[b])
            if n == 0:
                accepted.append(0)
                follow.append(-1)
                continue
            kids = lambda i: [j for j in range(i + 1, n) if self.parents[s + j] == i]  # noqa: E731
            order, rejected, drawn_from = [0], [], None
            while True:
                cur = order[-1]
                rejected, rest, taken = [], 1.0, None
                best = None
                if self.mode == "greedy":
                    best = int(self.x[s + cur].float().argmax())
                else:
                    p = self.probs(s + cur)
                for c in kids(cur):
                    token = int(self.tokens[s + c])
                    if not 0 <= token < self.vocab:
                        continue
                    if self.mode == "greedy":
                        if token == best:
                            taken = c
                            break
                        continue
                    u, pt = float(self.u[s + c]), float(p[token])
                    border = u * float(self.q[s + c, token]) if self.q is not None else u * rest
                    if token in [t for _, t in rejected]:
                        continue
                    assert pt == 0 or abs(border - pt) > near * pt, "inputs too near a border"
                    if pt > 0 and border < pt:
                        taken = c
                        break
                    rejected.append((c, token))
                    rest -= pt
                if taken is None:
                    break
                order.append(taken)
            accepted.append(len(order) - 1)
            path[s:s + n] = order + [-1] * (n - len(order))
            if self.mode == "greedy":
                follow.append(best if (self.x[s + cur] > -math.inf).any() else -1)
                continue
            left = p.clone()
            if self.q is not None:
                if rejected:
                    left = (p - self.q[s + rejected[-1][0]].double()).clamp(min=0)
            else:
                for _, t in rejected:
                    left[t] = 0
            if not (left > 0).any():
                left = p
            ratio = torch.where(self.noise[b] > 0, left / self.noise[b].double(), 0.0)
            two = ratio.topk(min(2, self.vocab)).values
            if self.vocab > 1 and float(two[0]) > 0:
                assert float(two[1]) < float(two[0]) * (1 - near), "inputs too near a border"
            follow.append(int(ratio.argmax()) if float(two[0]) > 0 else -1)
        return np.array(accepted), path, np.array(follow)


def good(case, status=0, **kw):
    got, flags = case.run(**kw)
    assert flags == status
    want = case.plain()
    for name, a, b in zip(("accepted", "path", "next_token"), got, want):
        np.testing.assert_array_equal(a, b, err_msg=name)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("mode,tree", [("greedy", False), ("greedy", True), ("lookup", False), ("lookup", True), ("drawn", False)])
@pytest.mark.parametrize("vocab,odd", [(1000, 0), (4099, 0), (32768, 0), (5001, 3)])
def test_modes_types_and_sizes(dtype, mode, tree, vocab, odd):
    good(VerifyCase(vocab + len(mode), [5, 1, 0, 9, 2, 16], vocab, dtype=dtype, mode=mode, tree=tree, odd=odd))


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("mode", ["greedy", "lookup"])
def test_tree_sizes(n, mode):
    good(VerifyCase(n, [n, max(0, n - 1), n], 2000, mode=mode, tree=True))


@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 255, 2047, 2049])
@pytest.mark.parametrize("mode", ["greedy", "lookup", "drawn"])
def test_small_vocabularies(vocab, mode):
    for dtype in ("f32", "bf16"):
        case = VerifyCase(vocab, [3, 4, 2], vocab, dtype=dtype, mode=mode)
        if mode == "drawn":  # (few entries, probabilities in 16 bits: a residual may be nothing but roundings)
            case.q = torch.softmax(torch.randn(case.q.shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV), -1).to(case.qt)
        good(case)


@pytest.mark.parametrize("mode,tree", [("lookup", True), ("drawn", False), ("greedy", False)])
@pytest.mark.parametrize("temp", [0.3, 1.7])
def test_masked_entries_temperatures_and_large_vocabularies(mode, tree, temp):
    good(VerifyCase(5, [9, 4], 200003, mode=mode, tree=tree, masked=True, temp=temp))
    good(VerifyCase(6, [9, 4, 17], 131072, dtype="bf16", mode=mode, tree=tree, temp=temp, draft_dtype="f32"))


@pytest.mark.parametrize("req", [320, 321, 700])
@pytest.mark.parametrize("mode", ["greedy", "lookup", "drawn"])
def test_many_requests(req, mode):
    counts = np.random.default_rng(req).integers(0, 4, req)
    good(VerifyCase(req, counts.tolist(), 5000, dtype="f16", mode=mode))


def test_the_same_token_twice_among_siblings():
    """The second is not tried again: its probability went with the first."""
    case = VerifyCase(7, [5], 500, tree=True)
    case.parents[:] = [-1, 0, 0, 0, 1]
    best = int(case.x[0].argmax())
    case.tokens[:] = [0, best, best, best, 3]
    for u in ([0.9999999, 0.0, 0.0], [0.0, 0.5, 0.5]):
        case.u[1:4] = torch.tensor(u, device=DEV)
        good(case)


def test_equal_largest_logits_and_ratios_go_to_the_lowest_id():
    case = VerifyCase(8, [2, 1], 3000, mode="greedy")
    case.x[0, [70, 900, 2500]] = 50.0
    case.tokens[1] = 70
    accepted, path, follow = good(case)
    assert accepted[0] == 1
    case.tokens[1] = 900
    assert good(case)[0][0] == 0
    case = VerifyCase(9, [1], 3000)
    case.x[0] = 1.0
    case.noise[0] = 1.0
    got, status = case.run()
    assert status == 0 and got[2][0] == 0
    case.noise[0, 1234] = case.noise[0, 77] = 0.5
    got, status = case.run()
    assert got[2][0] == 77


def test_draws_follow_the_target():
    """10,000 requests of one token and one draft: what comes first is distributed as the target says, within five
    standard deviations."""
    n, vocab = 10000, 8
    rng = np.random.default_rng(10)
    p = np.array([0.3, 0.25, 0.2, 0.1, 0.08, 0.05, 0.02, 0.0])
    q = np.array([0.05, 0.4, 0.1, 0.1, 0.2, 0.05, 0.1, 0.0])
    for mode in ("lookup", "drawn"):
        case = VerifyCase(10, [2] * n, vocab, mode="greedy")
        case.mode, case.inv = mode, 1.0
        case.x = torch.log(torch.tensor(p, device=DEV)).float().repeat(2 * n, 1)
        case.q = torch.tensor(q, device=DEV).float().repeat(2 * n, 1) if mode == "drawn" else None
        drafts = rng.choice(vocab, n, p=q)
        case.tokens = np.stack([np.zeros(n, np.int64), drafts], 1).reshape(-1)
        (accepted, _, follow), status = case.run()
        assert status == 0
        first = np.where(accepted == 1, drafts, follow)
        for x in range(vocab):
            assert abs((first == x).sum() - n * p[x]) <= 5 * math.sqrt(n * p[x] * (1 - p[x])) + 1e-9


def test_nothing_left_of_the_rest():
    """p and q alike, and a uniform number that rejects all the same: drawn from p."""
    case = VerifyCase(11, [2], 64, mode="drawn")
    case.x[0] = -math.inf
    case.x[0, 5] = case.x[0, 9] = 0.0
    case.q[1] = 0
    case.q[1, 5] = case.q[1, 9] = 0.5
    case.tokens[1] = 5
    case.u[1] = 1.0  # (outside [0, 1): rejects)
    got, status = case.run()
    assert status == 0 and got[0][0] == 0 and got[2][0] in (5, 9)
    case.noise[0, 9] = -1.0  # cannot be drawn
    assert case.run()[0][2][0] == 5
    # looked up: the only token that can occur, rejected
    case = VerifyCase(12, [2], 64)
    case.x[0] = -math.inf
    case.x[0, 5] = 0.0
    case.tokens[1], case.u[1] = 5, 1.0
    got, status = case.run()
    assert got[0][0] == 0 and got[2][0] == 5


def test_rows_without_entries_and_rows_that_are_not_finite():
    for mode in ("greedy", "lookup", "drawn"):
        case = VerifyCase(13, [3, 3, 3, 2], 900, mode=mode)
        case.x[0] = -math.inf          # nothing can occur behind the first row
        case.x[3, 100] = float("nan")  # with children
        case.x[6, 100] = float("inf")
        case.tokens[10] = int(case.x[9].argmax())
        case.u[10] = 0.0
        case.x[10, 5] = float("nan")   # a leaf, accepted
        got, status = case.run()
        assert status == mv.MOE_DEV_VALUE, mode
        assert got[0].tolist() == [0, 0, 0, 1] and got[2].tolist() == [-1, -1, -1, -1], mode


def test_bad_tokens_parents_and_lengths():
    case = VerifyCase(14, [4, 3], 700, tree=True)
    case.parents[:7] = [-1, 0, 0, 1, -1, 0, 1]
    case.tokens[1] = 700
    case.parents[6] = 2  # its own index: hangs on nothing
    got, status = case.run()
    assert status == mv.MOE_DEV_INDEX
    case.parents[6] = -1
    for a, b in zip(got, case.plain()):
        np.testing.assert_array_equal(a, b)
    case = VerifyCase(15, [3, 65, 2], 700)
    got, status = case.run()
    assert status == mv.MOE_DEV_LENGTH and got[0][1] == 0 and got[2][1] == -1 and (got[1][3:68] == -9).all()
    case = VerifyCase(16, [3, 4, 2], 700)
    for start in ([0, 9, 4, 9], [0, -3, 7, 9], [2**31 - 1, 0, 5, 9], [5, 3, 2, 2**31 - 1], [0, 3, 7, 10]):
        outs, flags = case.outputs(), word()
        args = case.args(outs, flags)
        case.keep[0].copy_(i32(start))
        ws = torch.zeros(mv.moe_verify_drafts_workspace_bytes(args), dtype=torch.uint8, device=DEV)
        mv.moe_verify_drafts(args, at(ws), ws.numel(), stream())
        assert int(flags.item()) & mv.MOE_DEV_LENGTH


def test_rows_of_nobody_are_left_as_they_were():
    case = VerifyCase(17, [3, 2], 1000, pad=4)
    got = good(case)
    assert (got[1][5:] == -9).all()


def test_no_rows_at_all():
    case = VerifyCase(18, [0, 0], 100)
    got, status = case.run()
    assert status == 0 and got[0].tolist() == [0, 0] and got[2].tolist() == [-1, -1]


def test_repeated_calls_and_one_workspace_for_many_shapes():
    cases = [VerifyCase(s, c, v, mode=m) for s, c, v, m in ((1, [8], 130000, "lookup"), (2, [2] * 400, 3000, "drawn"),
                                                          (3, [64, 3], 20000, "greedy"), (4, [7, 7], 130001, "drawn"))]
    ready = []
    for case in cases:
        outs, status = case.outputs(), word()
        ready.append((case, outs, status, case.args(outs, status), case.keep))
    ws = torch.zeros(max(mv.moe_verify_drafts_workspace_bytes(r[3]) for r in ready), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        for _, _, _, args, _ in ready:
            mv.moe_verify_drafts(args, at(ws), ws.numel(), stream())
    for case, outs, status, _, _ in ready:
        assert int(status.item()) == 0
        for a, b in zip(outs, case.plain()):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("mode", ["greedy", "lookup", "drawn"])
def test_a_replayed_graph_follows_contents_on_another_stream(mode):
    case = VerifyCase(19, [6, 3], 9000, mode=mode)
    outs, status = case.outputs(), word()
    args = case.args(outs, status)
    ws = torch.zeros(mv.moe_verify_drafts_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        mv.moe_verify_drafts(args, at(ws), ws.numel(), stream())
    for seed in (20, 21, 22):
        other = VerifyCase(seed, [6, 3], 9000, mode=mode)
        case.x.copy_(other.x)
        case.u.copy_(other.u)
        case.noise.copy_(other.noise)
        case.keep[2].copy_(i32(other.tokens))
        if mode == "drawn":
            case.q.copy_(other.q)
        case.tokens = other.tokens
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, case.plain()):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
    assert int(status.item()) == 0


@pytest.mark.parametrize("mode", ["greedy", "lookup", "drawn"])
def test_lengths_that_descend_bring_no_token_outside_the_vocabulary(mode):
    big = VerifyCase(60, [8, 8, 8], 4000, mode=mode)
    args = big.args(big.outputs(), word())
    ws = torch.zeros(mv.moe_verify_drafts_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    mv.moe_verify_drafts(args, at(ws), ws.numel(), stream())  # leaves sums and tokens of its own behind
    c = VerifyCase(61, [10, 4, 6], 100, mode=mode)
    c.start = np.array([0, 10, 5, 20])  # the third request's rows are partly the first's
    outs, status = c.outputs(), word()
    mv.moe_verify_drafts(c.args(outs, status), at(ws), ws.numel(), stream())
    accepted, path, follow = (t.cpu().numpy() for t in outs)
    assert int(status.item()) & mv.MOE_DEV_LENGTH
    assert accepted[1] == 0 and follow[1] == -1
    assert np.all((accepted >= 0) & (accepted < 15)) and np.all((follow >= -1) & (follow < 100))
    assert np.all((path >= -1) & (path < 15))


def test_greedy_trees_beside_draft_probabilities_that_are_not_read():
    case = VerifyCase(24, [6, 3, 0, 4], 3001, mode="greedy", tree=True)
    good(case, draft_probs=4096, draft_dtype=9, draft_stride=-4, noise_stride=-1)


@pytest.mark.parametrize("mode,tree", [("lookup", True), ("drawn", False)])
@pytest.mark.parametrize("size", [1e30, 1e34, 1e37])
def test_logits_and_temperatures_of_any_size(mode, tree, size):
    """Large logits at as large a temperature: the probabilities are those of ordinary ones."""
    case = VerifyCase(23, [9, 4, 1], 5003, mode=mode, tree=tree)
    case.x = case.x * size
    case.inv = float(np.float32(1 / size))
    good(case)


@pytest.mark.parametrize("first", [-2**31, -2**31 + 1, -2**31 + 5, -2**30, -1])
@pytest.mark.parametrize("mode", ["greedy", "lookup", "drawn"])
def test_row_starts_as_far_below_zero_as_they_go(mode, first):
    """The request that begins there, and the one that ends there, get nothing; the others what they get without them."""
    case = VerifyCase(27, [3, 4, 2, 5], 700, mode=mode)
    want = case.plain()
    outs, flags = case.outputs(), word()
    args = case.args(outs, flags)
    case.keep[0].copy_(i32([0, first, 7, 9, 14]))
    ws = torch.zeros(mv.moe_verify_drafts_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    mv.moe_verify_drafts(args, at(ws), ws.numel(), stream())
    accepted, path, follow = (t.cpu().numpy() for t in outs)
    assert int(flags.item()) == mv.MOE_DEV_LENGTH
    assert accepted[:2].tolist() == [0, 0] and follow[:2].tolist() == [-1, -1] and (path[:7] == -9).all()
    for got, expected, rows in ((accepted, want[0], slice(2, 4)), (path, want[1], slice(7, 14)), (follow, want[2], slice(2, 4))):
        np.testing.assert_array_equal(got[rows], expected[rows])


def test_greedy_rows_in_which_nothing_can_occur():
    """No token is the largest logit's, so no child stands, one of token 0 neither."""
    case = VerifyCase(28, [3, 2], 50, mode="greedy")
    case.x[0] = -math.inf
    case.tokens[1] = 0
    case.tokens[4] = int(case.x[3].argmax())
    got, status = case.run()
    assert status == 0 and got[0].tolist() == [0, 1] and got[1].tolist() == [0, -1, -1, 0, 1]
    assert got[2].tolist() == [-1, int(case.x[4].argmax())]
