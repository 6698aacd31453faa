"""Multi-axis rotary append (tv_kv_append_mrope) against the oracle: the
rotation's arithmetic is fixed to the rounding, so q, K and V are equal bit
for bit."""
import numpy as np
import pytest
import torch

import oracle
import serving_util as U
from gpu_util import bf16_bits, require_gpu
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200 import workloads as W
from paged_kv_cache_376_b200.device import bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu

FILL = 0x4040


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Case:
    def __init__(self, t, hq, hkv, axes, interleaved, seed, page_size=16,
                 max_position=8192):
        self.q = W._normal_bf16(seed, 2, (t, hq, 64))
        self.k = W._normal_bf16(seed, 3, (t, hkv, 64))
        self.v = W._normal_bf16(seed, 4, (t, hkv, 64))
        self.pos = U.multi_axis_positions(t, axes, max_position, seed)
        self.axis = U.pair_axes(axes, interleaved)
        self.table = U.rope_table(max_position)
        pages = -(-t // page_size) + 1
        self.slots = np.random.default_rng(seed).permutation(
            pages * page_size)[:t].astype(np.int32)
        self.pool = np.full((pages, page_size, hkv, 64), FILL, np.uint16)

    def expect(self):
        q, bad = oracle.mrope(self.q, self.pos, self.axis, self.table)
        k, _ = oracle.mrope(self.k, self.pos, self.axis, self.table)
        kp, vp, bad_slot = oracle.kv_append(k, self.v, self.slots, self.pool,
                                            self.pool)
        q = np.where((self.slots < 0)[:, None, None], FILL, q)
        return q, kp, vp, bad, bad_slot

    def run(self, fused=True, with_q=True, stream=None):
        t, hq, hkv = len(self.slots), self.q.shape[1], self.k.shape[1]
        if fused:
            rows = bf16_tensor(np.concatenate(
                [self.q, self.k, self.v], 1)).flatten(1)
            q, k, v = rows.split([hq * 64, hkv * 64, hkv * 64], 1)
            q, k, v = (x.unflatten(1, (-1, 64)) for x in (q, k, v))
        else:
            q, k, v = map(bf16_tensor, (self.q, self.k, self.v))
        kp, vp = bf16_tensor(self.pool), bf16_tensor(self.pool)
        q_out = bf16_tensor(np.full((t, hq, 64), FILL, np.uint16))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        _lib.tv_kv_append_mrope(
            q_out if with_q else None, q if with_q else None, k, v,
            i32_tensor(self.slots), i32_tensor(self.pos),
            i32_tensor(self.axis), kp, vp,
            torch.from_numpy(self.table).cuda(), err=err, stream=stream)
        torch.cuda.synchronize()
        return bf16_bits(q_out), bf16_bits(kp), bf16_bits(vp), int(err)

    def check(self, err=0, **kw):
        q, kp, vp, _, _ = self.expect()
        gq, gk, gv, ge = self.run(**kw)
        np.testing.assert_array_equal(gq, q)
        np.testing.assert_array_equal(gk, kp)
        np.testing.assert_array_equal(gv, vp)
        assert ge == err


@pytest.mark.parametrize("t", [1, 2, 7, 64, 333])
@pytest.mark.parametrize("heads", [(32, 8), (1, 1), (8, 1), (5, 3), (64, 16)])
@pytest.mark.parametrize("fused", [False, True])
def test_bit_exact(t, heads, fused):
    Case(t, *heads, 3, bool(t % 2), 600 + t).check(fused=fused)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("page_size", [16, 32])
def test_axes(axes, interleaved, page_size):
    Case(50, 8, 2, axes, interleaved, 620 + axes, page_size).check()


def test_a_long_call():
    Case(9000, 8, 2, 3, True, 630, max_position=20000).check()


def test_one_axis_is_the_single_axis_append():
    c = Case(100, 8, 2, 1, False, 631)
    _, gk, gv, _ = c.run()
    kp, vp = bf16_tensor(c.pool), bf16_tensor(c.pool)
    _lib.tv_kv_append_rope(bf16_tensor(c.k), bf16_tensor(c.v),
                           i32_tensor(c.slots), i32_tensor(c.pos[0]), kp, vp,
                           torch.from_numpy(c.table).cuda())
    np.testing.assert_array_equal(gk, bf16_bits(kp))
    np.testing.assert_array_equal(gv, bf16_bits(vp))


def test_padding_bad_slots_and_bad_positions():
    c = Case(40, 8, 2, 2, True, 632)
    c.slots[[3, 39]] = -1                        # padding: wholly skipped
    c.pos[0, 5], c.pos[1, 9] = -1, c.table.shape[0]
    c.pos[0, 3] = 1 << 30                        # of a padded token: unread
    c.check(err=_lib.DEVERR_BAD_POSITION)
    c.slots[7] = c.pool.shape[0] * 16 + 5
    c.check(err=_lib.DEVERR_BAD_POSITION | _lib.DEVERR_BAD_SLOT)
    c.pos[:] = 1
    c.axis[9] = 2                                # no such axis: none turn
    c.check(err=_lib.DEVERR_BAD_POSITION | _lib.DEVERR_BAD_SLOT)


def test_keys_alone():
    c = Case(20, 8, 2, 3, False, 633)
    _, kp, vp, _, _ = c.expect()
    q, gk, gv, err = c.run(with_q=False)
    assert (q == FILL).all() and err == 0
    np.testing.assert_array_equal(gk, kp)
    np.testing.assert_array_equal(gv, vp)


def test_in_place_on_contiguous_q():
    c = Case(70, 8, 2, 3, True, 634)
    q = bf16_tensor(c.q)
    kp, vp = bf16_tensor(c.pool), bf16_tensor(c.pool)
    _lib.tv_kv_append_mrope(q, q, bf16_tensor(c.k), bf16_tensor(c.v),
                            i32_tensor(c.slots), i32_tensor(c.pos),
                            i32_tensor(c.axis), kp, vp,
                            torch.from_numpy(c.table).cuda())
    np.testing.assert_array_equal(bf16_bits(q), c.expect()[0])


def test_captured_and_replayed_on_another_stream():
    c = Case(64, 8, 2, 3, True, 635)
    args = [bf16_tensor(c.q), bf16_tensor(c.k), bf16_tensor(c.v),
            i32_tensor(c.slots), i32_tensor(c.pos), i32_tensor(c.axis)]
    kp, vp = bf16_tensor(c.pool), bf16_tensor(c.pool)
    table = torch.from_numpy(c.table).cuda()
    out = torch.zeros_like(args[0])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        _lib.tv_kv_append_mrope(out, *args, kp, vp, table)
    c.pos = U.multi_axis_positions(64, 3, 8192, 9)
    args[4].copy_(i32_tensor(c.pos))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    q, ek, ev, _, _ = c.expect()
    np.testing.assert_array_equal(bf16_bits(out), q)
    np.testing.assert_array_equal(bf16_bits(kp), ek)
    np.testing.assert_array_equal(bf16_bits(vp), ev)


def test_refused_layouts():
    c = Case(8, 8, 2, 3, True, 636)
    args = [bf16_tensor(c.k), bf16_tensor(c.v), i32_tensor(c.slots),
            i32_tensor(c.pos), i32_tensor(c.axis), bf16_tensor(c.pool),
            bf16_tensor(c.pool), torch.from_numpy(c.table).cuda()]

    def call(q, out=None, **kw):
        a = list(args)
        for i, x in kw.items():
            a[int(i[1:])] = x
        _lib.tv_kv_append_mrope(torch.empty(8, 8, 64, dtype=torch.bfloat16,
                                            device="cuda")
                                if out is None else out, q, *a)

    q = bf16_tensor(c.q)
    call(q)
    with pytest.raises(ValueError):      # heads not contiguous
        call(q.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(_lib.TVError):    # token rows on odd strides
        call(torch.zeros(8, 8 * 64 + 4, dtype=torch.bfloat16, device="cuda")
             [:, :512].unflatten(1, (8, 64)))
    with pytest.raises(_lib.TVError):    # broadcast rows
        call(q[:1].expand(8, -1, -1))
    with pytest.raises(TypeError):
        call(q.float())
    with pytest.raises(ValueError):
        call(q, _3=args[3][:, :5].contiguous())
    with pytest.raises(ValueError):
        call(q, _4=args[4][:16].contiguous())
    with pytest.raises(ValueError):
        call(q[:5])
