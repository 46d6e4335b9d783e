"""The attention-side calls report their own launch: an error that some earlier call left with the runtime is not theirs."""
import ctypes
import re

import pytest
import torch

import spec_verify_layer_gb300 as mv
import syngen
from round_ops_helpers import DEV, MapCase, TreeCase, at, i32, stream, word

pytestmark = pytest.mark.gpu


def leave_an_error():
    """moe_last_device_status on a stream that is being captured: it cannot wait there, says so, and the runtime
    remembers."""
    rt = ctypes.CDLL(re.search(r"\S*libcudart\.so[.\d]*", open("/proc/self/maps").read()).group(0))
    side, graph = torch.cuda.Stream(), ctypes.c_void_p()
    cfg = syngen.CONFIGS["tiny"]
    handle = mv.moe_create(mv.make_dims(cfg.hidden, cfg.experts, cfg.top_k, cfg.inter, 4), 0)
    try:
        assert rt.cudaStreamBeginCapture(ctypes.c_void_p(side.cuda_stream), 1) == 0
        assert mv.moe_last_device_status(handle, side.cuda_stream) == mv.MOE_ECUDA
        rt.cudaStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph))
        rt.cudaGetLastError()
    finally:
        mv.moe_destroy(handle)


def test_an_earlier_error_is_not_reported_again():
    torch.cuda.synchronize()
    case = MapCase(1, [5, 9], [3, 4], 16)
    leave_an_error()
    _, status = case.run()
    assert status == 0

    tree = TreeCase(1, [40, 7], [3, 2], hq=4, hkv=2, d=64, page=16, dtype="bf16")
    leave_an_error()
    out, lse, status = tree.run()
    assert status == 0
    tree.check(out, lse)

    flag, x = word(), torch.randn((3, 1000), device=DEV)
    token, logp = i32([1, 2, 3]), torch.zeros(3, device=DEV)
    args = mv.make_logprob_args(n_rows=3, vocab=1000, dtype=mv.MOE_F32, logits=at(x), stride=1000, dev_status=at(flag),
                                tokens=at(token), logp=at(logp))
    ws = torch.zeros(mv.moe_token_logprobs_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    leave_an_error()
    mv.moe_token_logprobs(args, at(ws), ws.numel(), stream())
    assert torch.allclose(logp, torch.log_softmax(x, -1)[torch.arange(3), token.long()], atol=1e-4)

    q = torch.randn((2, 6, 64), device=DEV).bfloat16()
    cache, q_out = torch.zeros((2, 1, 16, 1, 64), dtype=torch.bfloat16, device=DEV), torch.zeros_like(q[:, :4])
    pos, slot = i32([3, 4]), i32([1, 2])
    rope = mv.make_qk_rope_args(
        n_rows=2, q_heads=4, kv_heads=1, head_dim=64, rot_dim=0, dtype=mv.MOE_BF16, q=at(q), k=at(q[:, 4:]), v=at(q[:, 5:]),
        q_stride=384, k_stride=384, v_stride=384, q_out=at(q_out), q_out_stride=256, row_pos=at(pos), row_slot=at(slot),
        dev_status=at(flag), cache=mv.make_kv_cache(at(cache[0]), at(cache[1]), n_pages=1, page_size=16, page_stride=1024,
                                                    slot_stride=64, head_stride=64))
    leave_an_error()
    mv.moe_qk_rope_cache(rope, stream())
    assert torch.equal(q_out, q[:, :4]) and torch.equal(cache[1, 0, 1:3, 0], q[:, 5]) and int(flag.item()) == 0
