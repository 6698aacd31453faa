"""Truncation and compaction of the device page pool, and whole-page copies,
bit for bit against the sequential model."""
import numpy as np
import pytest
import torch

import serving_util as U
from gpu_util import bf16_bits, require_gpu
from oracle.pool import PagePool, pages_for
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200.device import bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Pair:
    """The same pool on the GPU and in the model."""

    def __init__(self, num_pages, bt, ctx, page_size, hkv=1, seed=0):
        rng = np.random.default_rng(seed)
        self.n, self.ps = num_pages, page_size
        self.bt, self.ctx = bt.copy(), ctx.copy()
        self.kp = rng.integers(0, 1 << 16, (num_pages, page_size, hkv, 64)
                               ).astype(np.uint16)
        self.vp = self.kp[::-1].copy()
        self.pool = PagePool(num_pages, bt, ctx, page_size=page_size)
        self.g_bt, self.g_ctx = i32_tensor(bt), i32_tensor(ctx)
        self.g_kp, self.g_vp = bf16_tensor(self.kp), bf16_tensor(self.vp)
        self.state = _lib.pool_state(num_pages)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        _lib.tv_pool_init(self.state, block_tables=self.g_bt,
                          context_lens=self.g_ctx, page_size=page_size,
                          err=self.err)

    def check(self, err=0):
        torch.cuda.synchronize()
        st = self.state.cpu().numpy()
        n = self.n
        assert st[0] == self.pool.top
        np.testing.assert_array_equal(st[4:4 + st[0]], self.pool.stack)
        np.testing.assert_array_equal(st[4 + n:4 + 2 * n], self.pool.ref)
        assert not st[4 + 2 * n:4 + 4 * n].any()      # scratch at zero
        np.testing.assert_array_equal(self.g_bt.cpu().numpy(), self.bt)
        np.testing.assert_array_equal(self.g_ctx.cpu().numpy(), self.ctx)
        np.testing.assert_array_equal(bf16_bits(self.g_kp), self.kp)
        np.testing.assert_array_equal(bf16_bits(self.g_vp), self.vp)
        assert int(self.err) == err
        self.err.zero_()

    def truncate(self, new):
        self.pool.truncate(self.bt, self.ctx, new)
        _lib.tv_pool_truncate(self.state, self.g_bt, self.g_ctx,
                              i32_tensor(np.asarray(new)), err=self.err)

    def compact(self, copy="call"):
        moves, count = _lib.pool_moves(self.n)
        moves.fill_(-5)
        want = self.pool.compact(self.bt, self.ctx, self.kp, self.vp)
        pools = dict(k_pool=self.g_kp, v_pool=self.g_vp) \
            if copy == "call" else dict(page_size=self.ps)
        _lib.tv_pool_compact(self.state, self.g_bt, self.g_ctx, moves, count,
                             err=self.err, **pools)
        if copy != "call":
            _lib.tv_page_copy(self.g_kp, self.g_vp, moves[0], moves[1],
                              num_pairs=count, err=self.err)
        n = int(count)
        assert n == len(want)
        np.testing.assert_array_equal(
            moves[:, :n].cpu().numpy().T.reshape(-1, 2),
            np.asarray(want, np.int32).reshape(-1, 2))
        assert (moves[:, n:] == -5).all()


def _random(seed, num_pages, batch, page_size, **kw):
    bt, ctx = U.random_pool(seed, num_pages, batch, page_size, **kw)
    return Pair(num_pages, bt, ctx, page_size, seed=seed)


@pytest.mark.parametrize("page_size", [16, 32])
@pytest.mark.parametrize("num_pages,batch", [
    (1, 1), (33, 3), (100, 9), (1000, 100), (5000, 1024), (40000, 700)])
def test_truncate_and_compact(num_pages, batch, page_size):
    rng = np.random.default_rng(num_pages)
    p = _random(num_pages, num_pages, batch, page_size,
                width=12 if num_pages < 40000 else 40)
    p.check()
    for step in range(4):
        p.truncate([int(rng.integers(c // 2, c + 1)) for c in p.ctx])
        p.check()
        p.compact("call" if step % 2 else "lists")
        p.check()
    p.compact()                     # nothing to move
    p.check()
    p.truncate([0] * batch)         # a release of everything
    p.check()
    assert p.pool.top == num_pages
    p.compact()
    p.check()


def test_long_tables():
    """Rows of many hundred pages; pages of one row shared by all others."""
    n = 3000
    perm = np.random.default_rng(3).permutation(n)[:2500].astype(np.int32)
    bt = np.full((5, 2600), -1, np.int32)
    ctx = np.zeros(5, np.int64)
    for s, m in enumerate((2500, 2500, 1, 700, 0)):
        bt[s, :m] = perm[:m]
        ctx[s] = m * 16 - (s if m else 0)
    p = Pair(n, bt, ctx, 16)
    p.truncate([40000 - 17, 5, 1, 0, 0])
    p.check()
    p.compact()
    p.check()
    p.truncate([33, 5, 0, 0, 0])
    p.check()
    p.compact()
    p.check()


def test_truncate_refuses_lengths_one_by_one():
    bt, ctx = U.random_pool(5, 60, 6, 16)
    p = Pair(60, bt, ctx, 16)
    p.truncate([-1, int(ctx[1]) + 1, 0, 0, 1 << 30, int(ctx[5])])
    p.check(err=_lib.DEVERR_BAD_CONTEXT)


def test_truncate_flags_bad_pages():
    bt = np.array([[0, 1, 2], [3, 4, -1]], np.int32)
    p = Pair(8, bt, np.array([48, 32]), 16)
    p.g_bt[0, 2] = 8
    p.g_bt[1, 1] = -1
    _lib.tv_pool_truncate(p.state, p.g_bt, p.g_ctx, i32_tensor([16, 16]),
                          err=p.err)
    torch.cuda.synchronize()
    assert int(p.err) == _lib.DEVERR_BAD_PAGE
    st = p.state.cpu().numpy()
    assert st[0] == 4 and list(st[4:8]) == [7, 6, 5, 1]
    assert list(st[12:20]) == [1, 0, 1, 1, 1, 0, 0, 0]


def test_compact_of_another_page_size_changes_nothing():
    bt, ctx = U.random_pool(7, 60, 6, 16)
    p = Pair(60, bt, ctx, 16)
    moves, count = _lib.pool_moves(60)
    count.fill_(9)
    _lib.tv_pool_compact(p.state, p.g_bt, p.g_ctx, moves, count, page_size=32,
                         err=p.err)
    assert int(count) == 0
    p.check(err=_lib.DEVERR_BAD_SEQ)


def test_append_after_truncate_and_compact():
    """The pool that comes out serves on: appends pop the pages the model
    pops, with copy-on-write of a shared page cut in its middle."""
    bt = np.full((3, 8), -1, np.int32)
    bt[0, :5] = [30, 7, 29, 3, 11]
    bt[1, :5] = [30, 7, 29, 3, 12]
    bt[2, :2] = [20, 21]
    p = Pair(32, bt, np.array([75, 70, 20]), 16)
    p.truncate([60, 59, 18])
    p.compact()
    p.check()
    for n in ([1, 1, 1], [9, 0, 20]):
        p.pool.append_slots(p.bt, p.ctx, np.asarray(n), p.kp, p.vp)
        _lib.tv_pool_append_slots(p.state, p.g_bt, p.g_ctx, p.g_kp, p.g_vp,
                                  num_new_tokens=i32_tensor(n), err=p.err)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(p.g_bt.cpu().numpy(), p.bt)
        np.testing.assert_array_equal(bf16_bits(p.g_kp), p.kp)
        assert int(p.state[0]) == p.pool.top


@pytest.mark.parametrize("page_size,hkv", [(16, 1), (32, 8), (16, 3), (32, 5)])
def test_page_copy(page_size, hkv):
    n = 64
    rng = np.random.default_rng(hkv)
    kp = rng.integers(0, 1 << 16, (n, page_size, hkv, 64)).astype(np.uint16)
    vp = kp[::-1].copy()
    perm = rng.permutation(n)
    src, dst = perm[:24].astype(np.int32), perm[24:48].astype(np.int32)
    src[3], dst[9], src[11], dst[12] = -1, n, n + 7, -9
    good = [i for i in range(24) if i not in (3, 9, 11, 12)]
    for m in (None, 0, 10, 24, 99, -3):
        gk, gv = bf16_tensor(kp), bf16_tensor(vp)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        _lib.tv_page_copy(gk, gv, i32_tensor(src), i32_tensor(dst),
                          num_pairs=None if m is None else i32_tensor([m]),
                          err=err)
        used = min(max(24 if m is None else m, 0), 24)
        ek, ev = kp.copy(), vp.copy()
        for i in good:
            if i < used:
                ek[dst[i]], ev[dst[i]] = kp[src[i]], vp[src[i]]
        np.testing.assert_array_equal(bf16_bits(gk), ek)
        np.testing.assert_array_equal(bf16_bits(gv), ev)
        assert int(err) == (_lib.DEVERR_BAD_PAGE if used > 3 else 0)


def test_captured_compaction_replays_on_new_contents():
    bt, ctx = U.random_pool(11, 200, 20, 16)
    p = Pair(200, bt, ctx, 16)
    moves, count = _lib.pool_moves(200)
    new = i32_tensor(np.zeros(20))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        _lib.tv_pool_truncate(p.state, p.g_bt, p.g_ctx, new, err=p.err)
        _lib.tv_pool_compact(p.state, p.g_bt, p.g_ctx, moves, count, p.g_kp,
                             p.g_vp, err=p.err)
    rng = np.random.default_rng(1)
    for _ in range(3):
        want = [int(rng.integers(c // 2, c + 1)) for c in p.ctx]
        new.copy_(i32_tensor(want))
        g.replay()
        p.pool.truncate(p.bt, p.ctx, want)
        p.pool.compact(p.bt, p.ctx, p.kp, p.vp)
        p.check()


def test_captured_page_copies_follow_one_another():
    """A copy behind a memcpy, a copy that reads what the last one wrote, and a
    further layer's copy behind a compaction, in one graph."""
    n = 120
    bt, ctx = U.random_pool(12, n, 12, 16)
    p = Pair(n, bt, ctx, 16)
    moves, count = _lib.pool_moves(n)
    k2, v2 = p.g_kp.clone(), p.g_vp.clone()
    kp = np.random.default_rng(2).integers(
        0, 1 << 16, (n, 16, 2, 64)).astype(np.uint16)
    fresh = bf16_tensor(kp)
    gk, gv = torch.empty_like(fresh), torch.empty_like(fresh)
    a, b, c = (i32_tensor(np.arange(i, i + 40)) for i in (0, 40, 80))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        gv.copy_(fresh)
        gk.copy_(fresh)
        _lib.tv_page_copy(gk, gv, a, b, err=p.err)
        _lib.tv_page_copy(gk, gv, b, c, err=p.err)
        _lib.tv_pool_compact(p.state, p.g_bt, p.g_ctx, moves, count, p.g_kp,
                             p.g_vp, err=p.err)
        _lib.tv_page_copy(k2, v2, moves[0], moves[1], num_pairs=count,
                          err=p.err)
    p.pool.compact(p.bt, p.ctx, p.kp, p.vp)
    want = np.concatenate([kp[:40]] * 3)
    for _ in range(3):              # the second compaction finds nothing to move
        g.replay()
        np.testing.assert_array_equal(bf16_bits(gk), want)
        np.testing.assert_array_equal(bf16_bits(gv), want)
        np.testing.assert_array_equal(bf16_bits(k2), bf16_bits(p.g_kp))
        np.testing.assert_array_equal(bf16_bits(v2), bf16_bits(p.g_vp))
        p.check()


def test_pages_for_is_the_kernels_rounding():
    assert [pages_for(n, 16) for n in (0, 1, 16, 17)] == [0, 1, 1, 2]
