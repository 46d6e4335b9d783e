"""Refusals and sizes of the attention-side calls, on the host: every argument is checked before anything runs.

Only arguments that are refused are passed here, so no pointer is ever used.
"""
import ctypes

import pytest

import spec_verify_layer_gb300 as mv

P = 4096  # an aligned address that no refused call touches
INF, NAN = float("inf"), float("nan")


def fields(struct):
    return {name: kind for name, kind in struct._fields_}


def refused(fn, args, code, *rest):
    assert getattr(mv.lib(), fn)(None if args is None else ctypes.byref(args), *rest) == code


def map_args(**kw):
    d = dict(n_req=2, n_rows=8, page_size=16, n_pages=10, table_width=4, n_free=3, ctx_len=P, new_len=P, free_pages=P,
             block_table=P, row_start=P, pages=P, n_taken=P, row_req=P, row_pos=P, row_slot=P, dev_status=P)
    d.update(kw)
    return mv.make_map_args(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=0), mv.MOE_EINVAL), (dict(n_rows=-1), mv.MOE_EINVAL), (dict(page_size=0), mv.MOE_EINVAL),
    (dict(n_pages=0), mv.MOE_EINVAL), (dict(table_width=0), mv.MOE_EINVAL), (dict(n_free=-1), mv.MOE_EINVAL),
    (dict(ctx_len=None), mv.MOE_EINVAL), (dict(new_len=P + 2), mv.MOE_EINVAL), (dict(free_pages=0), mv.MOE_EINVAL),
    (dict(block_table=None), mv.MOE_EINVAL), (dict(row_start=None), mv.MOE_EINVAL), (dict(pages=None), mv.MOE_EINVAL),
    (dict(n_taken=None), mv.MOE_EINVAL), (dict(row_req=0), mv.MOE_EINVAL), (dict(row_pos=P + 4), mv.MOE_EINVAL),
    (dict(row_slot=0), mv.MOE_EINVAL), (dict(tree_mask=P + 8), mv.MOE_EINVAL), (dict(parents=P + 1), mv.MOE_EINVAL),
    (dict(dev_status=None), mv.MOE_EINVAL), (dict(dev_status=P + 1), mv.MOE_EINVAL),
    (dict(n_req=16385), mv.MOE_EUNSUPPORTED), (dict(page_size=65537), mv.MOE_EUNSUPPORTED),
    (dict(n_pages=1 << 27), mv.MOE_EUNSUPPORTED), (dict(table_width=1 << 30), mv.MOE_EUNSUPPORTED),
])
def test_round_map_refusals(kw, code):
    refused("moe_round_map", map_args(**kw), code, None)


def cache(**kw):
    d = dict(k=P, v=P, n_pages=4, page_size=16, page_stride=16 * 256, slot_stride=256, head_stride=128)
    d.update(kw)
    return mv.make_kv_cache(d.pop("k"), d.pop("v"), **d)


BAD_CACHES = [
    (dict(k=None), mv.MOE_EINVAL), (dict(v=P + 8), mv.MOE_EINVAL), (dict(n_pages=0), mv.MOE_EINVAL),
    (dict(page_size=0), mv.MOE_EINVAL), (dict(page_stride=12), mv.MOE_EINVAL), (dict(slot_stride=-8), mv.MOE_EINVAL),
    (dict(head_stride=1), mv.MOE_EINVAL), (dict(page_size=65537), mv.MOE_EUNSUPPORTED),
    (dict(n_pages=1 << 27), mv.MOE_EUNSUPPORTED),
]


def rope_args(**kw):
    d = dict(n_rows=3, q_heads=4, kv_heads=2, head_dim=128, rot_dim=64, dtype=mv.MOE_BF16, q=P, k=P, v=P, q_stride=1024,
             k_stride=1024, v_stride=1024, q_out=2 * P, q_out_stride=512, row_pos=P, row_slot=P, cache=cache(),
             dev_status=P, inv_freq=P, q_gain=P, k_gain=P)
    d.update(kw)
    return mv.make_qk_rope_args(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(n_rows=-1), mv.MOE_EINVAL), (dict(q_heads=0), mv.MOE_EINVAL), (dict(kv_heads=0), mv.MOE_EINVAL),
    (dict(head_dim=0), mv.MOE_EINVAL), (dict(head_dim=96), mv.MOE_EUNSUPPORTED),
    (dict(rot_dim=-16), mv.MOE_EINVAL), (dict(rot_dim=144), mv.MOE_EINVAL), (dict(rot_dim=24), mv.MOE_EUNSUPPORTED),
    (dict(dtype=mv.MOE_F32), mv.MOE_EUNSUPPORTED), (dict(dtype=7), mv.MOE_EINVAL),
    (dict(eps=-1e-6), mv.MOE_EINVAL), (dict(eps=NAN), mv.MOE_EINVAL), (dict(eps=INF), mv.MOE_EINVAL),
    (dict(rot_scale=NAN), mv.MOE_EINVAL), (dict(q=0), mv.MOE_EINVAL), (dict(k=P + 8), mv.MOE_EINVAL),
    (dict(v=0), mv.MOE_EINVAL), (dict(q_out=0), mv.MOE_EINVAL), (dict(q_stride=1028), mv.MOE_EINVAL),
    (dict(v_stride=-8), mv.MOE_EINVAL), (dict(q_out_stride=4), mv.MOE_EINVAL), (dict(q_gain=P + 4), mv.MOE_EINVAL),
    (dict(inv_freq=0), mv.MOE_EINVAL), (dict(inv_freq=P + 4), mv.MOE_EINVAL), (dict(row_pos=0), mv.MOE_EINVAL),
    (dict(row_slot=0), mv.MOE_EINVAL), (dict(dev_status=None), mv.MOE_EINVAL),
    (dict(q_out=P), mv.MOE_EINVAL),  # in place, but with another stride
    (dict(q_heads=257), mv.MOE_EUNSUPPORTED), (dict(kv_heads=257), mv.MOE_EUNSUPPORTED),
] + [(dict(cache=cache(**c)), code) for c, code in BAD_CACHES])
def test_qk_rope_refusals(kw, code):
    refused("moe_qk_rope_cache", rope_args(**kw), code, None)


def tree_args(**kw):
    d = dict(n_req=2, n_rows=8, max_tree=4, q_heads=8, kv_heads=2, head_dim=128, dtype=mv.MOE_F16, q=P, q_stride=1024,
             out=P, out_stride=1024, row_start=P, ctx_len=P, block_table=P, table_width=4, cache=cache(), scale=0.1,
             dev_status=P, tree_mask=P, lse=P)
    d.update(kw)
    return mv.make_tree_attention_args(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=0), mv.MOE_EINVAL), (dict(n_rows=-1), mv.MOE_EINVAL), (dict(max_tree=0), mv.MOE_EINVAL),
    (dict(max_tree=65), mv.MOE_EUNSUPPORTED), (dict(q_heads=7), mv.MOE_EINVAL), (dict(kv_heads=0), mv.MOE_EINVAL),
    (dict(q_heads=130, kv_heads=2), mv.MOE_EUNSUPPORTED), (dict(head_dim=80), mv.MOE_EUNSUPPORTED),
    (dict(dtype=mv.MOE_F32), mv.MOE_EUNSUPPORTED), (dict(dtype=-1), mv.MOE_EINVAL), (dict(scale=INF), mv.MOE_EINVAL),
    (dict(scale=NAN), mv.MOE_EINVAL), (dict(q=0), mv.MOE_EINVAL), (dict(out=P + 8), mv.MOE_EINVAL),
    (dict(q_stride=1020), mv.MOE_EINVAL), (dict(out_stride=-8), mv.MOE_EINVAL), (dict(row_start=None), mv.MOE_EINVAL),
    (dict(ctx_len=None), mv.MOE_EINVAL), (dict(block_table=None), mv.MOE_EINVAL), (dict(table_width=0), mv.MOE_EINVAL),
    (dict(tree_mask=P + 4), mv.MOE_EINVAL), (dict(lse=P + 2), mv.MOE_EINVAL), (dict(dev_status=None), mv.MOE_EINVAL),
    (dict(n_req=16385), mv.MOE_EUNSUPPORTED),
] + [(dict(cache=cache(**c)), code) for c, code in BAD_CACHES])
def test_tree_attention_refusals(kw, code):
    a = tree_args(**kw)
    assert mv.moe_tree_attention_workspace_bytes(a) == 0
    refused("moe_tree_attention", a, code, P, 1 << 40, None)


def logp_args(**kw):
    d = dict(n_rows=3, vocab=1000, dtype=mv.MOE_F32, logits=P, stride=1000, dev_status=P, tokens=P, top_k=4, logp=P,
             entropy=P, rank=P, top_ids=P, top_logp=P)
    d.update(kw)
    return mv.make_logprob_args(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(n_rows=-1), mv.MOE_EINVAL), (dict(vocab=0), mv.MOE_EINVAL), (dict(vocab=(1 << 24) + 1), mv.MOE_EUNSUPPORTED),
    (dict(top_k=-1), mv.MOE_EINVAL), (dict(top_k=33), mv.MOE_EUNSUPPORTED), (dict(dtype=3), mv.MOE_EINVAL),
    (dict(stride=-1), mv.MOE_EINVAL), (dict(logits=0), mv.MOE_EINVAL), (dict(logits=P + 2), mv.MOE_EINVAL),
    (dict(tokens=0), mv.MOE_EINVAL), (dict(tokens=0, logp=0), mv.MOE_EINVAL), (dict(top_ids=0), mv.MOE_EINVAL),
    (dict(top_logp=0), mv.MOE_EINVAL), (dict(logp=P + 1), mv.MOE_EINVAL), (dict(dev_status=None), mv.MOE_EINVAL),
    (dict(inv_temperature=0.0), mv.MOE_EINVAL), (dict(inv_temperature=-1.0), mv.MOE_EINVAL),
    (dict(inv_temperature=INF), mv.MOE_EINVAL), (dict(inv_temperature=NAN), mv.MOE_EINVAL),
])
def test_token_logprobs_refusals(kw, code):
    a = logp_args(**kw)
    assert mv.moe_token_logprobs_workspace_bytes(a) == 0
    refused("moe_token_logprobs", a, code, P, 1 << 40, None)


def test_missing_descriptor_and_workspace():
    for fn, rest in (("moe_round_map", (None,)), ("moe_qk_rope_cache", (None,)),
                     ("moe_tree_attention", (P, 1 << 40, None)), ("moe_token_logprobs", (P, 1 << 40, None))):
        refused(fn, None, mv.MOE_EINVAL, *rest)
    for fn, size, a in (("moe_tree_attention", mv.moe_tree_attention_workspace_bytes, tree_args()),
                        ("moe_token_logprobs", mv.moe_token_logprobs_workspace_bytes, logp_args())):
        need = size(a)
        assert need > 0
        refused(fn, a, mv.MOE_EINVAL, None, need, None)
        refused(fn, a, mv.MOE_EINVAL, P + 8, need, None)
        refused(fn, a, mv.MOE_EWORKSPACE, P, need - 1, None)


def test_errors_raise_with_their_code():
    with pytest.raises(mv.MoeError) as e:
        mv.moe_round_map(map_args(n_req=0), 0)
    assert e.value.code == mv.MOE_EINVAL
    with pytest.raises(mv.MoeError) as e:
        mv.moe_tree_attention(tree_args(), P, 0, 0)
    assert e.value.code == mv.MOE_EWORKSPACE


def test_a_logprob_workspace_serves_every_shape():
    """One size for all: a workspace made for the widest round is enough for narrower ones, and the other way round."""
    sizes = {mv.moe_token_logprobs_workspace_bytes(logp_args(n_rows=n, vocab=v, stride=v, dtype=t, top_k=k))
             for n in (0, 1, 5, 64, 65, 77, 152, 153, 5000) for v in (1, 1000, 131072, 1 << 24)
             for t in (mv.MOE_F32, mv.MOE_BF16) for k in (0, 32)}
    assert len(sizes) == 1 and sizes.pop() > 0


@pytest.mark.parametrize("held", [P - 4, P + 4, P - 4 * 255, P + 4 * 255])
def test_held_pages_partly_over_pages(held):
    """In place or apart (that a call in place runs is tested on the GPU)."""
    refused("moe_round_map", map_args(n_req=256, pages=P, pages_held=held), mv.MOE_EINVAL, None)


# products of counts and strides that pass 64 bits, or come round to something small there
WRAPPED_CACHES = [dict(n_pages=1 << 26, page_size=16, page_stride=1 << 38), dict(n_pages=(1 << 26) + 1, page_stride=1 << 39),
                  dict(page_size=65536, n_pages=8, slot_stride=(1 << 40) - 8),
                  dict(n_pages=(1 << 27) - 1, page_stride=(1 << 40) - 8, slot_stride=(1 << 40) - 8)]


@pytest.mark.parametrize("kw", WRAPPED_CACHES)
def test_caches_whose_offsets_pass_64_bits(kw):
    a = tree_args(cache=cache(**kw))
    assert mv.moe_tree_attention_workspace_bytes(a) == 0
    refused("moe_tree_attention", a, mv.MOE_EUNSUPPORTED, P, 1 << 40, None)
    if kw.get("page_size") != 65536:  # (2^56 elements: an address space would hold them)
        refused("moe_qk_rope_cache", rope_args(cache=cache(**kw)), mv.MOE_EUNSUPPORTED, None)


@pytest.mark.parametrize("name", ["q_stride", "k_stride", "v_stride", "q_out_stride"])
def test_rows_whose_offsets_pass_64_bits(name):
    refused("moe_qk_rope_cache", rope_args(n_rows=1 << 24, **{name: (1 << 40) - 8}), mv.MOE_EUNSUPPORTED, None)


def test_logits_whose_offsets_pass_64_bits():
    a = logp_args(n_rows=1 << 24, stride=(1 << 40) - 1)
    assert mv.moe_token_logprobs_workspace_bytes(a) == 0
    refused("moe_token_logprobs", a, mv.MOE_EUNSUPPORTED, P, 1 << 40, None)


@pytest.mark.parametrize("width,page,ok", [(131067, 64, True), (131068, 64, False), (8388287, 1, True), (8388288, 1, True),
                                           (8388289, 1, False), (2**31 - 1, 65536, False)])
def test_the_limit_of_the_attentions_list(width, page, ok):
    """n_req * kv_heads * (table_width * page_size / 64, rounded up, + 4) below 2^31: up to 131,071 for 16,384 requests."""
    a = tree_args(n_req=16384, q_heads=1, kv_heads=1, table_width=width, cache=cache(page_size=page))
    assert (mv.moe_tree_attention_workspace_bytes(a) > 0) == ok
    if not ok:
        refused("moe_tree_attention", a, mv.MOE_EUNSUPPORTED, P, 1 << 40, None)


def test_a_list_whose_length_passes_64_bits():
    a = tree_args(n_req=16384, q_heads=1024, kv_heads=1024, table_width=2**31 - 1, cache=cache(page_size=65536, n_pages=8))
    assert mv.moe_tree_attention_workspace_bytes(a) == 0
