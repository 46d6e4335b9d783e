"""Refusals and sizes of the 8-bit cache's calls and of the verification, on the host."""
import math

import pytest

import spec_verify_layer_gb300 as mv
from test_round_ops_host import INF, NAN, P, refused


def cache8(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=4, page_size=16, block_size=8, format=mv.MOE_E4M3, page_stride=16 * 256,
             slot_stride=256, head_stride=128, scale_page_stride=4, scale_block_stride=2, scale_head_stride=1)
    d.update(kw)
    return mv.make_kv_cache8(d.pop("k"), d.pop("v"), d.pop("k_scale"), d.pop("v_scale"), **d)


BAD_CACHES = [
    (dict(k=None), mv.MOE_EINVAL), (dict(v=P + 8), mv.MOE_EINVAL), (dict(k_scale=None), mv.MOE_EINVAL),
    (dict(v_scale=P + 2), mv.MOE_EINVAL), (dict(n_pages=0), mv.MOE_EINVAL), (dict(page_size=0), mv.MOE_EINVAL),
    (dict(block_size=0), mv.MOE_EINVAL), (dict(block_size=3), mv.MOE_EINVAL), (dict(block_size=32), mv.MOE_EINVAL),
    (dict(page_size=24, block_size=16), mv.MOE_EINVAL), (dict(page_size=24, block_size=12), mv.MOE_EINVAL),
    (dict(format=mv.MOE_BF16), mv.MOE_EINVAL), (dict(format=9), mv.MOE_EINVAL), (dict(page_stride=24), mv.MOE_EINVAL),
    (dict(slot_stride=-16), mv.MOE_EINVAL), (dict(head_stride=8), mv.MOE_EINVAL), (dict(scale_head_stride=-1), mv.MOE_EINVAL),
    (dict(scale_page_stride=1 << 40), mv.MOE_EINVAL), (dict(page_size=256, block_size=256), mv.MOE_EUNSUPPORTED),
    (dict(page_size=65544), mv.MOE_EUNSUPPORTED), (dict(n_pages=1 << 27), mv.MOE_EUNSUPPORTED),
]


def rows_args(**kw):
    d = dict(n_req=2, n_rows=8, kv_heads=2, head_dim=128, dtype=mv.MOE_BF16, k=P, v=P, k_stride=256, v_stride=256, row_start=P,
             ctx_len=P, block_table=P, table_width=4, cache=cache8(), dev_status=P)
    d.update(kw)
    return mv.make_cache8_args(**d)


@pytest.mark.parametrize("fn", ["moe_cache8_append", "moe_cache8_read"])
@pytest.mark.parametrize("kw,code", [
    (dict(n_req=0), mv.MOE_EINVAL), (dict(n_rows=-1), mv.MOE_EINVAL), (dict(table_width=0), mv.MOE_EINVAL),
    (dict(kv_heads=0), mv.MOE_EINVAL), (dict(head_dim=0), mv.MOE_EINVAL), (dict(head_dim=96), mv.MOE_EUNSUPPORTED),
    (dict(dtype=mv.MOE_E4M3), mv.MOE_EINVAL), (dict(k=0), mv.MOE_EINVAL), (dict(v=P + 8), mv.MOE_EINVAL),
    (dict(k_stride=252), mv.MOE_EINVAL), (dict(v_stride=-8), mv.MOE_EINVAL), (dict(row_start=None), mv.MOE_EINVAL),
    (dict(ctx_len=P + 2), mv.MOE_EINVAL), (dict(block_table=None), mv.MOE_EINVAL), (dict(dev_status=None), mv.MOE_EINVAL),
    (dict(n_req=16385), mv.MOE_EUNSUPPORTED), (dict(n_rows=(1 << 24) + 1), mv.MOE_EUNSUPPORTED),
    (dict(kv_heads=257), mv.MOE_EUNSUPPORTED),
] + [(dict(cache=cache8(**c)), code) for c, code in BAD_CACHES])
def test_rows_refusals(fn, kw, code):
    refused(fn, rows_args(**kw), code, None)


def attn_args(**kw):
    d = dict(n_req=2, n_rows=8, max_tree=4, q_heads=8, kv_heads=2, head_dim=128, dtype=mv.MOE_BF16, q=P, q_stride=1024, out=P,
             out_stride=1024, row_start=P, ctx_len=P, block_table=P, table_width=4, cache=cache8(), scale=0.1, dev_status=P)
    d.update(kw)
    return mv.make_tree_attention8_args(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=0), mv.MOE_EINVAL), (dict(n_rows=-1), mv.MOE_EINVAL), (dict(max_tree=0), mv.MOE_EINVAL),
    (dict(max_tree=65), mv.MOE_EUNSUPPORTED), (dict(q_heads=7), mv.MOE_EINVAL), (dict(kv_heads=0), mv.MOE_EINVAL),
    (dict(q_heads=130, kv_heads=2), mv.MOE_EUNSUPPORTED), (dict(head_dim=32), mv.MOE_EUNSUPPORTED),
    (dict(dtype=mv.MOE_F32), mv.MOE_EUNSUPPORTED), (dict(dtype=mv.MOE_E4M3), mv.MOE_EINVAL), (dict(scale=NAN), mv.MOE_EINVAL),
    (dict(scale=INF), mv.MOE_EINVAL), (dict(q=P + 8), mv.MOE_EINVAL), (dict(out=0), mv.MOE_EINVAL),
    (dict(q_stride=1020), mv.MOE_EINVAL), (dict(out_stride=-8), mv.MOE_EINVAL), (dict(lse=P + 2), mv.MOE_EINVAL),
    (dict(tree_mask=P + 4), mv.MOE_EINVAL), (dict(dev_status=None), mv.MOE_EINVAL), (dict(n_rows=(1 << 20) + 1), mv.MOE_EUNSUPPORTED),
    (dict(cache=cache8(n_pages=65, page_stride=1 << 30)), mv.MOE_EUNSUPPORTED),
] + [(dict(cache=cache8(**c)), code) for c, code in BAD_CACHES])
def test_attention_refusals(kw, code):
    args = attn_args(**kw)
    refused("moe_tree_attention8", args, code, P, 1 << 30, None)
    assert mv.moe_tree_attention8_workspace_bytes(args) == 0


def test_attention_workspace():
    args = attn_args()
    size = mv.moe_tree_attention8_workspace_bytes(args)
    assert size > 0
    refused("moe_tree_attention8", args, mv.MOE_EINVAL, None, size, None)
    refused("moe_tree_attention8", args, mv.MOE_EINVAL, P + 8, size, None)
    refused("moe_tree_attention8", args, mv.MOE_EWORKSPACE, P, size - 1, None)


def verify_args(**kw):
    d = dict(n_req=2, n_rows=8, vocab=1000, dtype=mv.MOE_BF16, logits=P, stride=1000, row_start=P, tokens=P, uniform=P, noise=P,
             noise_stride=1000, accepted=P, path=P, next_token=P, dev_status=P)
    d.update(kw)
    return mv.make_verify_args(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=0), mv.MOE_EINVAL), (dict(n_rows=-1), mv.MOE_EINVAL), (dict(vocab=0), mv.MOE_EINVAL),
    (dict(inv_temperature=0.0), mv.MOE_EINVAL), (dict(inv_temperature=-1.0), mv.MOE_EINVAL), (dict(inv_temperature=NAN), mv.MOE_EINVAL),
    (dict(dtype=mv.MOE_I8), mv.MOE_EINVAL), (dict(draft_probs=P, draft_dtype=7), mv.MOE_EINVAL), (dict(stride=-1), mv.MOE_EINVAL),
    (dict(noise_stride=-1), mv.MOE_EINVAL), (dict(draft_probs=P, draft_stride=-4), mv.MOE_EINVAL), (dict(logits=0), mv.MOE_EINVAL),
    (dict(logits=P + 1), mv.MOE_EINVAL), (dict(tokens=0), mv.MOE_EINVAL), (dict(uniform=0), mv.MOE_EINVAL), (dict(noise=0), mv.MOE_EINVAL),
    (dict(noise=P + 2), mv.MOE_EINVAL), (dict(accepted=None), mv.MOE_EINVAL), (dict(path=0), mv.MOE_EINVAL),
    (dict(next_token=P + 2), mv.MOE_EINVAL), (dict(dev_status=None), mv.MOE_EINVAL), (dict(parents=P + 1), mv.MOE_EINVAL),
    (dict(draft_probs=P + 2), mv.MOE_EINVAL), (dict(parents=P, draft_probs=P), mv.MOE_EUNSUPPORTED),
    (dict(n_req=16385), mv.MOE_EUNSUPPORTED), (dict(n_rows=(1 << 20) + 1), mv.MOE_EUNSUPPORTED), (dict(vocab=(1 << 24) + 1), mv.MOE_EUNSUPPORTED),
])
def test_verify_refusals(kw, code):
    args = verify_args(**kw)
    refused("moe_verify_drafts", args, code, P, 1 << 30, None)
    assert mv.moe_verify_drafts_workspace_bytes(args) == 0


def test_verify_workspace():
    args = verify_args()
    size = mv.moe_verify_drafts_workspace_bytes(args)
    assert size > 0
    refused("moe_verify_drafts", args, mv.MOE_EINVAL, P + 8, size, None)
    refused("moe_verify_drafts", args, mv.MOE_EWORKSPACE, P, size - 1, None)
    # greedy needs neither random numbers nor drafts' probabilities
    assert mv.moe_verify_drafts_workspace_bytes(verify_args(inv_temperature=math.inf, uniform=0, noise=0)) > 0


def test_nothing_is_refused_as_null():
    for fn, rest in (("moe_cache8_append", (None,)), ("moe_cache8_read", (None,)), ("moe_tree_attention8", (P, 1 << 30, None)),
                     ("moe_verify_drafts", (P, 1 << 30, None))):
        refused(fn, None, mv.MOE_EINVAL, *rest)


def test_verify_workspace_does_not_fall_as_sizes_grow():
    """Sized once for a program's largest round it serves every smaller one, of any type of logits and drafts."""
    def size(**kw):
        return mv.moe_verify_drafts_workspace_bytes(verify_args(**kw))

    vocabs = [1, 1000, 4095, 4096, 8191, 8192, 16384, 32000, 32003, 65536, 129283, 131072, 262144, 1 << 24]
    rows = [0, 1, 2, 46, 47, 93, 94, 187, 188, 375, 661, 749, 750, 1499, 1500, 2999, 3000, 5999, 6001, 1 << 20]
    reqs = [1, 2, 9, 10, 18, 19, 24, 37, 38, 64, 75, 76, 151, 152, 303, 304, 320, 321, 700, 16384]
    kinds = [(mv.MOE_F32, 1.0), (mv.MOE_BF16, 1.0), (mv.MOE_F16, math.inf)]
    for req in (1, 24, 64, 320, 700):
        table = [[size(n_req=req, n_rows=r, vocab=v) for v in vocabs] for r in rows]
        for r, line in zip(rows, table):
            assert line == sorted(line), (req, r)
            for v, s in zip(vocabs, line):
                assert all(size(n_req=req, n_rows=r, vocab=v, dtype=t, inv_temperature=inv) == s for t, inv in kinds)
        for column in zip(*table):
            assert list(column) == sorted(column)
    for v in vocabs:
        column = [size(n_req=n, n_rows=661, vocab=v) for n in reqs]
        assert column == sorted(column), v


def test_greedy_does_not_look_at_what_it_does_not_read():
    """Random numbers and drafts' probabilities may be anything, also beside a tree."""
    greedy = dict(inv_temperature=math.inf, parents=P, draft_probs=P + 1, draft_dtype=9, draft_stride=-4, uniform=P + 2, noise=P + 1,
                  noise_stride=-1)
    size = mv.moe_verify_drafts_workspace_bytes(verify_args(inv_temperature=math.inf, parents=P))
    assert size > 0 and mv.moe_verify_drafts_workspace_bytes(verify_args(**greedy)) == size
    refused("moe_verify_drafts", verify_args(**greedy), mv.MOE_EWORKSPACE, P, size - 1, None)


@pytest.mark.parametrize("kw", [dict(scale_page_stride=0), dict(scale_block_stride=0), dict(scale_head_stride=0), dict(page_stride=0),
                                dict(slot_stride=0), dict(head_stride=0), dict(k_scale=P, v_scale=P)])
def test_append_refuses_caches_whose_blocks_share_places(kw):
    own = dict(k=P, v=2 * P, k_scale=3 * P, v_scale=4 * P)
    refused("moe_cache8_append", rows_args(cache=cache8(**{**own, **kw}), n_rows=0), mv.MOE_EINVAL, None)
    refused("moe_cache8_append", rows_args(cache=cache8(**own), n_rows=0), mv.MOE_OK, None)  # (no rows: nothing is touched)
    refused("moe_cache8_read", rows_args(cache=cache8(**{**own, **kw}), n_rows=0), mv.MOE_OK, None)
    # one of a kind needs no stride
    alone = {**own, "n_pages": 1, "page_size": 8, "page_stride": 0, "scale_page_stride": 0, "scale_block_stride": 0, "head_stride": 0,
             "scale_head_stride": 0}
    refused("moe_cache8_append", rows_args(cache=cache8(**alone), kv_heads=1, n_rows=0), mv.MOE_OK, None)
