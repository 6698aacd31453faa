"""Chunk and cross attention over the paged cache against the oracle.

Bound (assert_parity): the output's own rounding is at most 2^-8 of it.  The
weights come from binary32 scores of 64 products (relative error of a weight
at most 64 x 2^-23 x sum|q k| x scale x log2 e, about 2^-14 here) and enter the
second product with 16 bits (2^-17) where a block's first row sees fewer than
512 keys; with |v| < 6 that is below 1e-3, the absolute part.  From 512 keys on
they enter with 8 bits: an element is off by sum p d v / sum p with |d| <= 2^-8
(half a step of bf16), independent and evenly spread, so with standard deviation
at most 2^-8 / sqrt(3) x sqrt(sum p^2 v^2) / sum p.  For normal scores of
deviation 1 sum p^2 / (sum p)^2 is e / n, so that is at most 2.26e-3 x
sqrt(e / 512) = 1.6e-4, and 1e-3 is six of them.  Where few keys carry the
weight, the bound is 2^-8 x sum p |v| / sum p (test_concentrated_weights)."""
import numpy as np
import pytest
import torch

import oracle
import serving_util as U
from gpu_util import (assert_parity, bf16_bits, err_word, gpu_append,
                      grow_keys, oracle_after_append, require_gpu, upload)
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _call(db, scale, causal=True, maxq=None, workspace=True, out=None,
          stream=None, q=None):
    q = db.q if q is None else q
    out = torch.empty_like(q) if out is None else out
    if maxq is None:
        maxq = int(db.query_start_loc.diff().max())
    ws = workspace or None if isinstance(workspace, bool) else workspace
    if ws is True:
        ws = _lib.chunk_workspace(db.context_lens.numel(), maxq, q.shape[1],
                                  db.k_pool.shape[2])
    fn = _lib.tv_paged_chunk if causal else _lib.tv_paged_cross_attention
    fn(out, q, db.query_start_loc, db.k_pool, db.v_pool, db.block_tables,
       db.context_lens, scale, maxq, workspace=ws, err=db.err, stream=stream)
    return out


def _heads(group, hkv=4):
    return dict(num_q_heads=hkv * group, num_kv_heads=hkv)


def _chunk(prefixes, chunks, seed, **kw):
    wl = W.prefill_workload(prefixes, chunks, seed=seed, **kw)
    db = upload(wl)
    gpu_append(db)
    kp, vp = oracle_after_append(wl)
    ref = oracle.paged_prefill(wl.q, wl.query_start_loc, kp, vp,
                               wl.block_tables, wl.context_lens, wl.scale)
    return wl, db, ref


def _cross(lens, rows, seed, **kw):
    wl = U.cross_workload(lens, rows, seed, **kw)
    db = upload(wl)
    ref = oracle.paged_cross(wl.q, wl.query_start_loc, wl.k_pool, wl.v_pool,
                             wl.block_tables, wl.context_lens, wl.scale)
    return wl, db, ref


RAGGED = ([0, 15, 16, 1, 100, 333, 7, 64], [1, 1, 3, 17, 2, 8, 0, 33])


@pytest.mark.parametrize("page_size", [16, 32])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("workspace", [False, True])
def test_chunk_every_row(page_size, group, workspace):
    wl, db, ref = _chunk(*RAGGED, 501, page_size=page_size, **_heads(group))
    out = _call(db, wl.scale, workspace=workspace)
    assert_parity(out, ref, "chunk")
    assert err_word(db) == 0


@pytest.mark.parametrize("page_size", [16, 32])
@pytest.mark.parametrize("group", [1, 4, 8])
@pytest.mark.parametrize("prefixes,chunks", [
    ([0], [200]), ([31, 500], [129, 257]), ([0, 2000, 63], [513, 1, 300]),
], ids=["prompt", "ragged", "mixed"])
def test_long_chunks(page_size, group, prefixes, chunks):
    wl, db, ref = _chunk(prefixes, chunks, 502, page_size=page_size,
                         **_heads(group, 2))
    for ws in (False, True):
        assert_parity(_call(db, wl.scale, workspace=ws), ref, "long chunk")
    assert err_word(db) == 0


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 8, 13, 16, 31])
@pytest.mark.parametrize("group", [1, 4, 8])
def test_draft_lengths(rows, group):
    wl, db, ref = _chunk([300, 0, 1000], [rows] * 3, 503, **_heads(group))
    assert_parity(_call(db, wl.scale), ref, "draft")
    # a larger bound on the rows gives the same
    assert_parity(_call(db, wl.scale, maxq=rows + 100), ref, "draft")
    assert err_word(db) == 0


@pytest.mark.parametrize("lens", [
    [20000], [20000, 3, 9000, 1], [5000] * 3 + [17] * 40 + [12000],
], ids=["one", "few", "many"])
@pytest.mark.parametrize("rows", [1, 4, 9, 70])
def test_long_contexts_split_over_keys(lens, rows):
    chunks = [min(rows, n) for n in lens]
    wl, db, ref = _chunk([n - t for n, t in zip(lens, chunks)], chunks, 504,
                         num_q_heads=8, num_kv_heads=2)
    assert_parity(_call(db, wl.scale), ref, "split")
    assert_parity(_call(db, wl.scale, workspace=False), ref, "unsplit")
    # the order in which splits finish leaves no trace in the result
    a = bf16_bits(_call(db, wl.scale))
    for _ in range(5):
        np.testing.assert_array_equal(bf16_bits(_call(db, wl.scale)), a)
    assert err_word(db) == 0


@pytest.mark.parametrize("rows,group", [(1, 1), (5, 4), (29, 1), (60, 1),
                                        (90, 4)])
def test_one_kv_head_in_many_parts(rows, group):
    """One long sequence spread over the whole GPU beside a short one: more
    parts than a warp joins at once, in both kernels."""
    lens = [60000, 130]
    wl, db, ref = _chunk([n - rows for n in lens], [rows] * 2, 517,
                         num_q_heads=group, num_kv_heads=1)
    a = _call(db, wl.scale)
    assert_parity(a, ref, "many parts")
    assert torch.equal(a, _call(db, wl.scale))
    assert err_word(db) == 0


@pytest.mark.parametrize("page_size", [16, 32])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("lens,rows", [
    ([1500, 0, 1, 15, 16, 17, 700], [1] * 7),
    ([0, 40, 333, 2, 64], [5, 300, 1, 130, 0]),
    ([9000, 31], [3, 70]),
], ids=["step", "prompt", "long"])
def test_cross_every_row(page_size, group, lens, rows):
    wl, db, ref = _cross(lens, rows, 505, page_size=page_size,
                         **_heads(group, 2))
    for ws in (False, True):
        out = _call(db, wl.scale, causal=False, workspace=ws)
        assert_parity(out, ref, "cross")
    assert err_word(db) == 0


@pytest.mark.parametrize("rows", [8, 200])
def test_climbing_maxima(rows):
    """Row maxima that grow along the context: the running offset moves again
    and again.  The weights' error grows with the scores (up to 2^6 times
    those above), so only |v| x 2^-8 is asked beside the output's rounding."""
    wl = grow_keys(W.prefill_workload([900, 200], [rows, rows], seed=506,
                                      **_heads(4, 2)))
    db = upload(wl)
    gpu_append(db)
    kp, vp = oracle_after_append(wl)
    ref = oracle.paged_prefill(wl.q, wl.query_start_loc, kp, vp,
                               wl.block_tables, wl.context_lens, wl.scale)
    for ws in (False, True):
        assert_parity(_call(db, wl.scale, workspace=ws), ref, "climbing",
                      abs_=6 * 2.0 ** -8)


@pytest.mark.parametrize("rows,causal", [(8, True), (200, True), (8, False),
                                         (200, False)])
def test_concentrated_weights(rows, causal):
    """Scores of deviation 6 over 2000 keys: a few keys carry each row.  The
    worst case of 8-bit weights, half a step of bf16, is 2^-8 of the sum of
    p |v| (taken from the oracle with |V|), beside the output's 2^-8 and the
    weights' binary32 error: 64 additions x 2^-24 x sum|q k| (about 41) x scale
    x log2 e (1.08) x ln 2 = 1.2e-4 of p |v|, doubled for the sum: < 2^-10."""
    lens = [2000, 700]
    wl = (W.prefill_workload([n - rows for n in lens], [rows] * 2, seed=516,
                             **_heads(4, 2)) if causal
          else U.cross_workload(lens, [rows] * 2, 516, **_heads(4, 2)))
    db = upload(wl)
    if causal:
        gpu_append(db)
        kp, vp = oracle_after_append(wl)
    else:
        kp, vp = wl.k_pool, wl.v_pool
    fn = oracle.paged_prefill if causal else oracle.paged_cross
    scale = 6 * wl.scale
    ref, size = (fn(wl.q, wl.query_start_loc, kp, v, wl.block_tables,
                    wl.context_lens, scale)
                 for v in (vp, vp & np.uint16(0x7fff)))
    for ws in (False, True):
        got = W.bf16_to_f64(bf16_bits(_call(db, scale, causal, workspace=ws)))
        bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * size
        assert (np.abs(got - ref) <= bound).all()
    assert err_word(db) == 0


def test_rows_behind_the_last_sequence_stay():
    for causal in (True, False):
        wl, db, ref = (_chunk([40, 9], [5, 70], 507) if causal
                       else _cross([40, 9], [5, 70], 507))
        n = ref.shape[0]
        q = torch.cat([db.q, db.q[:9]])
        out = torch.full_like(q, 7.0)
        _call(db, wl.scale, causal=causal, out=out, q=q)
        assert_parity(out[:n], ref, "real rows")
        assert (out[n:] == 7.0).all()
        assert err_word(db) == 0


@pytest.mark.parametrize("rows", [6, 150])
def test_later_keys_are_hidden_whatever_they_hold(rows):
    """The K of the last new tokens is set to NaN and their V to infinity:
    earlier rows, which do not see them, keep their values bit for bit, and
    rows that see them lose theirs."""
    for group in (1, 4, 8):
        wl, db, ref = _chunk([21, 50], [rows, rows], 508, **_heads(group, 2))
        before = _call(db, wl.scale)
        cut = rows - 3
        kf = db.k_pool.view(-1, *db.k_pool.shape[2:])
        vf = db.v_pool.view(-1, *db.v_pool.shape[2:])
        for s in (0, 1):
            slots = db.slot_mapping[s * rows + cut:(s + 1) * rows].long()
            vf[slots, :, 5] = float("inf")
            vf[slots, :, 40] = float("nan")
        out = _call(db, wl.scale).view(2, rows, -1, 64)
        b = before.view(2, rows, -1, 64)
        assert torch.equal(out[:, :cut], b[:, :cut])
        hit = torch.zeros(64, dtype=torch.bool, device="cuda")
        hit[[5, 40]] = True
        assert not out[:, cut:][..., hit].isfinite().any()
        assert out[:, cut:][..., ~hit].isfinite().all()
        for s in (0, 1):
            slots = db.slot_mapping[s * rows + cut:(s + 1) * rows].long()
            kf[slots] = float("nan")
        out = _call(db, wl.scale).view(2, rows, -1, 64)
        assert torch.equal(out[:, :cut], b[:, :cut])
        assert out[:, cut:].isnan().all()


def test_a_row_of_nan_stays_its_own():
    for causal in (True, False):
        wl, db, ref = (_chunk([40, 300], [5, 90], 509) if causal
                       else _cross([40, 300], [5, 90], 509))
        before = _call(db, wl.scale, causal=causal)
        db.q[[2, 50], 3] = float("nan")
        out = _call(db, wl.scale, causal=causal)
        assert out[[2, 50], 3].isnan().all()
        out[[2, 50], 3] = before[[2, 50], 3]
        assert torch.equal(out, before)


def test_bad_pages_are_flagged_and_left_out():
    wl = W.prefill_workload([100, 40, 0], [70, 3, 20], seed=510)
    db = upload(wl)
    gpu_append(db)
    kp, vp = oracle_after_append(wl)
    bt = wl.block_tables.copy()
    bt[0, 2] = wl.num_pages + 5
    bt[1, 0] = -3
    bt[2, 0] = wl.num_pages
    db.block_tables.copy_(torch.from_numpy(bt))
    ref = oracle.paged_prefill(wl.q, wl.query_start_loc, kp, vp, bt,
                               wl.context_lens, wl.scale, allow_bad=True)
    for ws in (False, True):
        db.err.zero_()
        out = _call(db, wl.scale, workspace=ws)
        assert err_word(db) == _lib.DEVERR_BAD_PAGE
        first = int(wl.query_start_loc[2])
        assert not np.any(ref[first:first + 16])
        assert_parity(out, ref, "bad pages")


def test_sequences_with_impossible_rows_are_skipped():
    wl, db, ref = _chunk([20, 30, 40], [4, 5, 6], 511)
    # more rows than keys
    db.context_lens[1] = 4
    out = torch.full_like(db.q, 7.0)
    _call(db, wl.scale, out=out)
    assert err_word(db) == _lib.DEVERR_BAD_QUERY
    assert (out[4:9] == 7.0).all()
    assert_parity(out[:4], ref[:4], "others")
    assert_parity(out[9:], ref[9:], "others")
    # more rows than max_query_len; rows outside q
    db.context_lens[1] = 35
    for edit in ("maxq", "rows"):
        db.err.zero_()
        out.fill_(7.0)
        if edit == "maxq":
            _call(db, wl.scale, out=out, maxq=5)
        else:
            qsl = db.query_start_loc.clone()
            qsl[3] = 16
            db.query_start_loc.copy_(qsl)
            _call(db, wl.scale, out=out, maxq=8)
        assert err_word(db) == _lib.DEVERR_BAD_QUERY
        assert_parity(out[:9], ref[:9], "others")
        assert (out[9:] == 7.0).all()


def test_contexts_out_of_range_are_flagged_and_clamped():
    wl, db, _ = _cross([48, 48], [2, 3], 512)
    cap = wl.max_blocks_per_seq * wl.page_size
    db.context_lens.copy_(torch.tensor([-4, cap + 9], dtype=torch.int32))
    out = _call(db, wl.scale, causal=False)
    assert err_word(db) == _lib.DEVERR_BAD_CONTEXT
    assert not out[:2].any()
    ref = oracle.paged_cross(wl.q, wl.query_start_loc, wl.k_pool, wl.v_pool,
                             wl.block_tables, [0, cap], wl.scale)
    assert_parity(out, ref, "clamped")


@pytest.mark.parametrize("causal", [True, False])
def test_two_streams_and_graphs(causal):
    """Two calls at once with workspaces of their own, captured and replayed
    with other inputs."""
    make = _chunk if causal else _cross
    cases = [make([9000, 100], [4, 4], 513), make([6000, 64], [9, 200], 514)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs, graphs, wss = [], [], []
    for (wl, db, ref), st in zip(cases, streams):
        maxq = int(db.query_start_loc.diff().max())
        ws = _lib.chunk_workspace(2, maxq, db.q.shape[1], db.k_pool.shape[2])
        out = torch.empty_like(db.q)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            _call(db, wl.scale, causal, maxq, ws, out)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            _call(db, wl.scale, causal, maxq, ws, out)
        outs.append(out), graphs.append(g), wss.append(ws)
    for flip in (False, True):
        for (wl, db, ref), out in zip(cases, outs):
            out.zero_()
            if flip:
                db.q.neg_(), db.k_pool.neg_()      # the same scores
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for (wl, db, ref), out in zip(cases, outs):
            assert_parity(out, ref, "replay")
            assert err_word(db) == 0


def test_chunk_of_one_row_is_decode_and_prefill():
    lens = [1, 40, 777, 5000]
    wl, db, ref = _chunk([n - 1 for n in lens], [1] * 4, 515)
    out = _call(db, wl.scale)
    dec = torch.empty_like(db.q)
    _lib.tv_paged_decode(dec, db.q, db.k_pool, db.v_pool, db.block_tables,
                         db.context_lens, wl.scale, err=db.err)
    assert_parity(out, ref, "chunk")
    assert_parity(dec, ref, "decode")
    assert err_word(db) == 0
