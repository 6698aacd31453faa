"""Truncation and compaction of a pool of more pages than the compaction's
bitmap holds in shared memory (131,072): the bit words then go through the
state's scratch words, which have to be zero again afterwards.  Tables and
moves only; bit for bit against the sequential model."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu
from oracle.pool import PagePool
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200.device import i32_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("num_pages", [131072, 131073, 140001, 300000])
def test_compact_and_truncate(num_pages):
    rng = np.random.default_rng(num_pages)
    batch, width = 64, 1500
    perm = rng.permutation(num_pages)
    bt = np.full((batch, width), -1, np.int32)
    ctx = np.zeros(batch, np.int64)
    at = 0
    for s in range(batch):
        n = int(rng.integers(0, width + 1))
        bt[s, :n] = perm[at:at + n]
        at += n
        ctx[s] = max(0, 16 * n - int(rng.integers(0, 16)))
    model = PagePool(num_pages, bt, ctx)
    g_bt, g_ctx = i32_tensor(bt), i32_tensor(ctx)
    state = _lib.pool_state(num_pages)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _lib.tv_pool_init(state, block_tables=g_bt, context_lens=g_ctx, err=err)

    def check():
        st = state.cpu().numpy()
        assert int(err) == 0
        assert st[0] == model.top
        np.testing.assert_array_equal(st[4:4 + st[0]], model.stack)
        np.testing.assert_array_equal(st[4 + num_pages:4 + 2 * num_pages],
                                      model.ref)
        assert not st[4 + 2 * num_pages:4 + 4 * num_pages].any()
        np.testing.assert_array_equal(g_bt.cpu().numpy(), bt)
        np.testing.assert_array_equal(g_ctx.cpu().numpy(), ctx)

    check()
    for step in range(2):
        moves, count = _lib.pool_moves(num_pages)
        moves.fill_(-5)
        want = model.compact(bt, ctx)
        _lib.tv_pool_compact(state, g_bt, g_ctx, moves, count, page_size=16,
                             err=err)
        n = int(count)
        assert n == len(want)
        assert n > 0 or step
        np.testing.assert_array_equal(
            moves[:, :n].cpu().numpy().T, np.asarray(want).reshape(-1, 2))
        assert (moves[:, n:] == -5).all()
        check()
        new = [int(rng.integers(0, c + 1)) for c in ctx]
        model.truncate(bt, ctx, new)
        _lib.tv_pool_truncate(state, g_bt, g_ctx, i32_tensor(new), err=err)
        check()
