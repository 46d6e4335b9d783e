"""moe_qk_rope_cache against the norm and the rotation in 64 bits.

Bound of an element: half a step of its type, and 4e-6 of the magnitude of its pair for the 32-bit work: the sum
of squares (at most 256 terms in a tree of 8 + 5 levels, 13 * 2^-24), root, division and two products (5 * 2^-24),
the cosine and sine (4e-7 for the 32-bit fraction of a turn, its rounding and sincospi) and the rotation (3 * 2^-24).
"""
import numpy as np
import pytest
import torch

import spec_verify_layer_gb300 as mv
from round_ops_helpers import DEV, DT, at, rotate64, stream, word

pytestmark = pytest.mark.gpu
SPECIAL = 777.0


class Rope:
    def __init__(self, seed, rows, hq, hkv, d, rot, dtype, *, interleaved=False, norm=(True, True), page=16,
                 layout="nhd", pos=None, scale=1.0, eps=1e-6, amp=1.5):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.dt, self.code = DT[dtype]
        self.hq, self.hkv, self.d, self.rot, self.inter, self.page = hq, hkv, d, rot, interleaved, page
        self.scale, self.eps, self.rows = scale, eps, rows
        self.qkv = (torch.randn((rows, hq + 2 * hkv + 1, d), generator=gen, device=DEV) * amp).to(self.dt)
        self.q, self.k, self.v = self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:hq + 2 * hkv]
        self.gain = [(1 + 0.3 * torch.randn(d, generator=gen, device=DEV)).to(self.dt) if n else None for n in norm]
        self.inv = 1e4 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / max(rot, 1))
        n_pages = rows // page + 2
        self.slots = n_pages * page
        shape = (n_pages, page, hkv, d) if layout == "nhd" else (n_pages, hkv, page, d)
        self.caches = [torch.full(shape, SPECIAL, dtype=self.dt, device=DEV) for _ in range(2)]
        if layout == "hnd":
            self.caches = [c.transpose(1, 2) for c in self.caches]
        self.slot = torch.from_numpy(np.random.default_rng(seed).permutation(self.slots)[:rows].astype(np.int32)).to(DEV)
        self.pos = torch.randint(0, 40000, (rows,), generator=gen, device=DEV, dtype=torch.int32) if pos is None else (
            torch.tensor(pos, dtype=torch.int32, device=DEV))

    def run(self, q_out=None):
        c = self.caches[0]
        out = torch.full((self.rows, self.hq, self.d), SPECIAL, dtype=self.dt, device=DEV) if q_out is None else q_out
        status = word()
        cache = mv.make_kv_cache(at(c), at(self.caches[1]), n_pages=c.shape[0], page_size=self.page,
                                 page_stride=c.stride(0), slot_stride=c.stride(1), head_stride=c.stride(2))
        args = mv.make_qk_rope_args(
            n_rows=self.rows, q_heads=self.hq, kv_heads=self.hkv, head_dim=self.d, rot_dim=self.rot, dtype=self.code,
            q=at(self.q), k=at(self.k), v=at(self.v), q_stride=self.q.stride(0), k_stride=self.k.stride(0),
            v_stride=self.v.stride(0), q_out=at(out), q_out_stride=out.stride(0), row_pos=at(self.pos),
            row_slot=at(self.slot), cache=cache, dev_status=at(status), inv_freq=at(self.inv) if self.rot else 0,
            q_gain=at(self.gain[0]), k_gain=at(self.gain[1]), interleaved=self.inter, eps=self.eps,
            rot_scale=self.scale)
        mv.moe_qk_rope_cache(args, stream())
        return out, int(status.item())

    def want(self, x, gain):
        return rotate64(x, gain, self.pos, self.inv, self.rot, self.inter, self.eps, self.scale)

    def near(self, got, ref):
        y, amp = ref
        u = torch.finfo(self.dt).eps / 2
        bound = u * y.abs() + 4e-6 * (1 + u) * amp + (2**-25 if self.dt == torch.float16 else 0)
        bad = ~((got.double() - y).abs() <= bound)
        assert not bad.any(), (int(bad.sum()), float((got.double() - y).abs().max()))

    def check(self, q_out, q_ref, k_ref):
        self.near(q_out, q_ref)
        ok = (self.slot >= 0) & (self.slot < self.slots)
        s = self.slot[ok].long()
        page, off = s // self.page, s % self.page
        self.near(self.caches[0][page, off], tuple(t[ok] for t in k_ref))
        assert torch.equal(self.caches[1][page, off], self.v[ok])
        rest = torch.ones(self.caches[0].shape[:2], dtype=torch.bool, device=DEV)
        rest[page, off] = False
        for c in self.caches:
            assert (c[rest] == SPECIAL).all()

    def refs(self):
        return self.want(self.q, self.gain[0]), self.want(self.k, self.gain[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 0), (128, 128), (128, 32), (128, 96), (256, 256), (256, 64),
                                   (256, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 1, 1), (3, 5, 1), (37, 12, 4)])
def test_rope(dtype, d, rot, interleaved, rows, hq, hkv):
    layout, page = ("hnd", 24) if rows == 3 else ("nhd", 16)
    r = Rope(d + rot + rows, rows, hq, hkv, d, rot, dtype, interleaved=interleaved, layout=layout, page=page)
    q_ref, k_ref = r.refs()
    out, status = r.run()
    assert status == 0
    r.check(out, q_ref, k_ref)


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
def test_without_norms(norm):
    r = Rope(1, 9, 6, 2, 128, 128, "bf16", norm=norm)
    refs = r.refs()
    out, status = r.run()
    assert status == 0
    r.check(out, *refs)


def test_many_rows_and_scale():
    r = Rope(2, 6001, 8, 2, 64, 32, "f16", scale=1.25, page=64)
    refs = r.refs()
    out, status = r.run()
    assert status == 0
    r.check(out, *refs)


def test_far_positions_keep_their_angles():
    """The reference's angle in 64 bits is itself off by 2^-53 of it: 2.4e-7 rad at 2^31; the kernel's by 3e-6."""
    pos = [0, 1, 2**20 - 1, 10**6, 2**24 + 1, -5]
    r = Rope(3, len(pos), 4, 2, 128, 128, "f16", pos=pos)
    refs = r.refs()
    out, status = r.run()
    assert status == 0
    r.check(out, *refs)
    r = Rope(3, 2, 4, 2, 128, 128, "bf16", pos=[2**31 - 1, -2**31])
    refs = r.refs()
    out, _ = r.run()
    r.check(out, *refs)


def test_frequencies_of_more_than_a_turn_and_negative_ones():
    r = Rope(4, 7, 2, 1, 64, 64, "f16", pos=[0, 1, 2, 3, 1000, 1001, 4096])
    r.inv = torch.linspace(-20.0, 20.0, 32, device=DEV, dtype=torch.float64)
    refs = r.refs()
    out, status = r.run()
    assert status == 0
    r.check(out, *refs)


def test_in_place():
    r = Rope(5, 21, 6, 2, 128, 64, "bf16")
    refs = r.refs()
    out, status = r.run(q_out=r.q)
    assert status == 0
    r.check(out, *refs)


def test_rows_without_a_slot_and_slots_outside_the_cache():
    r = Rope(6, 8, 4, 2, 64, 64, "bf16")
    refs = r.refs()
    r.slot[2] = -1
    out, status = r.run()
    assert status == 0
    r.check(out, *refs)
    r = Rope(6, 8, 4, 2, 64, 64, "bf16")
    refs = r.refs()
    r.slot[1], r.slot[5], r.slot[6] = r.slots, -2, 2**31 - 1
    out, status = r.run()
    assert status == mv.MOE_DEV_INDEX
    r.check(out, *refs)


def test_zero_rows_and_large_and_small_values():
    r = Rope(7, 0, 4, 2, 64, 64, "bf16")
    out, status = r.run()
    assert status == 0 and (r.caches[0] == SPECIAL).all()
    for amp, dtype in ((1e-3, "f16"), (1e3, "bf16"), (0.0, "bf16")):
        r = Rope(8, 5, 4, 2, 128, 128, dtype, amp=amp)
        refs = r.refs()
        out, status = r.run()
        r.check(out, *refs)


def test_one_bad_head_stays_alone():
    """An infinity or NaN in one head of one row changes no other head."""
    r = Rope(9, 6, 4, 2, 128, 128, "bf16")
    clean, _ = r.run()
    clean_k = r.caches[0].clone()
    r.q[3, 1, 5] = float("inf")
    r.k[2, 0, 7] = float("nan")
    out, _ = r.run()
    other = torch.ones((6, 4), dtype=torch.bool, device=DEV)
    other[3, 1] = False
    assert torch.equal(out[other], clean[other]) and not torch.isfinite(out[3, 1]).all()
    s = int(r.slot[2])
    now, was = r.caches[0], clean_k
    now[s // r.page, s % r.page, 0] = 0
    was[s // r.page, s % r.page, 0] = 0
    assert torch.equal(now, was)


def test_offsets_past_32_bits():
    """The last slots of a cache of more than 2^32 elements."""
    page, d, hkv = 256, 128, 1
    n_pages = (2**32 // (page * d)) + 2
    r = Rope(10, 3, 2, hkv, d, d, "bf16", page=page)
    k = torch.zeros(n_pages * page * d, dtype=torch.bfloat16, device=DEV).view(n_pages, page, hkv, d)
    r.caches = [k, torch.zeros_like(k)]
    r.slots = n_pages * page
    r.slot = torch.tensor([n_pages * page - 1, 5, n_pages * page - page - 3], dtype=torch.int32, device=DEV)
    refs = r.refs()
    out, status = r.run()
    assert status == 0
    r.near(out, refs[0])
    s = r.slot.long()
    r.near(k[s // page, s % page], refs[1])
    assert torch.equal(r.caches[1][s // page, s % page], r.v)
