"""The serving operators together, as a speculative step of a multimodal decoder
uses them: room for the drafts (tv_pool_append_slots), rotation and append of
two layers (tv_kv_append_mrope), attention of the drafts over the cache and over
the encoder's states (tv_paged_chunk, tv_paged_cross_attention), return of the
rejected drafts' pages (tv_pool_truncate), now and then a compaction with the
second layer's pages (tv_pool_compact, tv_page_copy).  Integers and pools equal
the model's bit for bit; attention is held to the parity bound."""
import numpy as np
import pytest
import torch

import oracle
import serving_util as U
from gpu_util import assert_parity, bf16_bits, require_gpu
from oracle.pool import PagePool
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200 import workloads as W
from paged_kv_cache_376_b200.device import bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu

HQ, HKV, AXES, MAX_POS, B = 8, 2, 3, 4096, 7


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("page_size", [16, 32])
def test_speculative_steps(page_size):
    rng = np.random.default_rng(page_size)
    bt, ctx = U.random_pool(5, 70, B, page_size, width=6)
    bt = np.concatenate([bt, np.full((B, 6), -1, np.int32)], 1)
    pool = PagePool(70, bt, ctx, page_size=page_size)
    layers = [[W._normal_bf16(layer, i, (70, page_size, HKV, 64))
               for i in (0, 1)] for layer in (40, 41)]
    enc = U.cross_workload([33, 0, 300, 1, 64, 16, 7], [1] * B, 43,
                           page_size=page_size, num_q_heads=HQ,
                           num_kv_heads=HKV)
    table = U.rope_table(MAX_POS)
    axis = U.pair_axes(AXES, True)
    g_bt, g_ctx = i32_tensor(bt), i32_tensor(ctx)
    g_layers = [[bf16_tensor(p) for p in kv] for kv in layers]
    g_enc = [bf16_tensor(enc.k_pool), bf16_tensor(enc.v_pool),
             i32_tensor(enc.block_tables), i32_tensor(enc.context_lens)]
    g_table, g_axis = torch.from_numpy(table).cuda(), i32_tensor(axis)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = _lib.pool_state(70)
    _lib.tv_pool_init(state, block_tables=g_bt, context_lens=g_ctx, err=err,
                      page_size=page_size)
    moves, count = _lib.pool_moves(70)
    ws = _lib.chunk_workspace(B, 6, HQ, HKV)

    for step in range(6):
        n_new = rng.integers(0, 7, B).astype(np.int32)
        # layer 0's pools see the copy-on-write of the append; the step
        # mirrors it into layer 1 with the pages that changed
        before = bt.copy()
        slots, served = pool.append_slots(bt, ctx, n_new, *layers[0])
        g_slots = torch.full((max(1, int(n_new.sum())),), -1,
                             dtype=torch.int32, device="cuda")
        _lib.tv_pool_append_slots(state, g_bt, g_ctx, *g_layers[0],
                                  num_new_tokens=i32_tensor(n_new),
                                  slot_mapping=g_slots, err=err)
        cow = [(before[s, b], bt[s, b]) for s in range(B)
               for b in range(bt.shape[1])
               if before[s, b] >= 0 and before[s, b] != bt[s, b]]
        if cow:
            src, dst = (i32_tensor(np.array(x)) for x in zip(*cow))
            _lib.tv_page_copy(*g_layers[1], src, dst, err=err)
            for a, b in cow:
                for p in layers[1]:
                    p[b] = p[a]
        new = np.where(served, n_new, 0)
        t = int(new.sum())
        assert len(slots) == t
        if t == 0:
            continue
        np.testing.assert_array_equal(g_slots[:t].cpu().numpy(), slots)
        qsl = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pos = U.multi_axis_positions(t, AXES, MAX_POS, step)
        g_qsl = i32_tensor(qsl)
        for kv, g_kv in zip(layers, g_layers):
            rows = W._normal_bf16(50 + step, 9, (t, HQ + 2 * HKV, 64))
            q, k, v = np.split(rows, [HQ, HQ + HKV], 1)
            fused = bf16_tensor(rows)
            g_q = torch.empty(t, HQ, 64, dtype=torch.bfloat16, device="cuda")
            _lib.tv_kv_append_mrope(
                g_q, fused[:, :HQ], fused[:, HQ:HQ + HKV], fused[:, HQ + HKV:],
                g_slots[:t], i32_tensor(pos), g_axis, *g_kv, g_table, err=err)
            q, _ = oracle.mrope(q, pos, axis, table)
            k, _ = oracle.mrope(k, pos, axis, table)
            kv[:] = oracle.kv_append(k, v, np.asarray(slots, np.int32),
                                     *kv)[:2]
            np.testing.assert_array_equal(bf16_bits(g_q), q)
            out, cross = torch.empty_like(g_q), torch.empty_like(g_q)
            _lib.tv_paged_chunk(out, g_q, g_qsl, *g_kv, g_bt, g_ctx, 0.125, 6,
                                workspace=ws, err=err)
            _lib.tv_paged_cross_attention(
                cross, g_q, g_qsl, *g_enc, 0.125, 6, workspace=ws, err=err)
            assert_parity(out, oracle.paged_prefill(
                q, qsl, *kv, bt, ctx, 0.125), "chunk")
            assert_parity(cross, oracle.paged_cross(
                q, qsl, enc.k_pool, enc.v_pool, enc.block_tables,
                enc.context_lens, 0.125), "cross")
        keep = [int(c - rng.integers(0, m + 1)) for c, m in zip(ctx, new)]
        pool.truncate(bt, ctx, keep)
        _lib.tv_pool_truncate(state, g_bt, g_ctx, i32_tensor(np.array(keep)),
                              err=err)
        if step % 2:
            want = pool.compact(bt, ctx, *layers[0])
            for a, b in want:
                for p in layers[1]:
                    p[b] = p[a]
            _lib.tv_pool_compact(state, g_bt, g_ctx, moves, count,
                                 *g_layers[0], err=err)
            _lib.tv_page_copy(*g_layers[1], moves[0], moves[1],
                              num_pairs=count, err=err)
        np.testing.assert_array_equal(g_bt.cpu().numpy(), bt)
        np.testing.assert_array_equal(g_ctx.cpu().numpy(), ctx)
        st = state.cpu().numpy()
        assert list(st[4:4 + st[0]]) == pool.stack
        for kv, g_kv in zip(layers, g_layers):
            for p, g in zip(kv, g_kv):
                np.testing.assert_array_equal(bf16_bits(g), p)
    # (a step may find the pool or a table row full: that is flagged)
    assert int(err) & ~(_lib.DEVERR_POOL_EMPTY | _lib.DEVERR_BAD_CONTEXT) == 0


def test_the_python_and_the_direct_route_agree():
    """Calls on the current stream are made in C++, calls with a stream of
    their own through ctypes: the same call either way."""
    wl = W.prefill_workload([100, 9], [5, 8], seed=61)
    kp, vp = bf16_tensor(wl.k_pool).nan_to_num(), \
        bf16_tensor(wl.v_pool).nan_to_num()
    q, qsl = bf16_tensor(wl.q), i32_tensor(wl.query_start_loc)
    bt, ctx = i32_tensor(wl.block_tables), i32_tensor(wl.context_lens)
    ws = _lib.chunk_workspace(2, 8, 32, 8)
    here = torch.cuda.current_stream()
    for fn in (_lib.tv_paged_chunk, _lib.tv_paged_cross_attention):
        a, b = torch.zeros_like(q), torch.zeros_like(q)
        fn(a, q, qsl, kp, vp, bt, ctx, 0.125, 8, workspace=ws)
        fn(b, q, qsl, kp, vp, bt, ctx, 0.125, 8, workspace=ws, stream=here)
        assert torch.equal(a, b) and a.any()
    t = q.shape[0]
    pos = i32_tensor(U.multi_axis_positions(t, 3, 64, 0))
    axis = i32_tensor(U.pair_axes(3, False))
    tab = torch.from_numpy(U.rope_table(64)).cuda()
    res = []
    for stream in (None, here):
        k2, v2, o = kp.clone(), vp.clone(), torch.zeros_like(q)
        _lib.tv_kv_append_mrope(o, q, bf16_tensor(wl.k_new),
                                bf16_tensor(wl.v_new),
                                i32_tensor(wl.slot_mapping), pos, axis, k2,
                                v2, tab, stream=stream)
        res.append((o, k2, v2))
    assert all(torch.equal(x, y) for x, y in zip(*res))
    n, res = wl.num_pages, []
    for stream in (None, here):
        st, b2, c2 = _lib.pool_state(n), bt.clone(), ctx.clone()
        k2, v2 = kp.clone(), vp.clone()
        moves, count = _lib.pool_moves(n)
        _lib.tv_pool_init(st, block_tables=b2, context_lens=c2)
        _lib.tv_pool_truncate(st, b2, c2, i32_tensor([50, 3]), stream=stream)
        _lib.tv_pool_compact(st, b2, c2, moves, count, k2, v2, stream=stream)
        _lib.tv_page_copy(k2, v2, moves[0], moves[1], num_pairs=count,
                          stream=stream)
        res.append((st, b2, c2, k2, v2, moves, count))
    assert all(torch.equal(x, y) for x, y in zip(*res))
    # what the direct route does not take is still said in Python's words
    with pytest.raises(TypeError, match="q must be"):
        _lib.tv_paged_chunk(a, q.float(), qsl, kp, vp, bt, ctx, 0.125, 8)
    with pytest.raises(_lib.TVError):
        _lib.tv_paged_chunk(a, q, qsl, kp, vp, bt, ctx, -1.0, 8)
    with pytest.raises(ValueError, match="shape mismatch"):
        _lib.tv_paged_chunk(a, q, qsl[:2], kp, vp, bt, ctx, 0.125, 8)
