"""Values of chunk and cross attention where the weights themselves show: two
keys that nearly cancel, and keys whose scores are minus infinity."""
import numpy as np
import pytest
import torch

import oracle
import serving_util as U
from gpu_util import (assert_parity, bf16_bits, err_word, require_gpu, upload)
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _bits(x):
    return W.bf16_bits(np.asarray(x, np.float32))


def _run(wl, causal, workspace):
    db = upload(wl)
    maxq = int(np.diff(wl.query_start_loc).max())
    ws = None
    if workspace:
        ws = _lib.chunk_workspace(len(wl.context_lens), maxq, wl.q.shape[1],
                                  wl.k_pool.shape[2])
    fn = _lib.tv_paged_chunk if causal else _lib.tv_paged_cross_attention
    out = torch.empty_like(db.q)
    fn(out, db.q, db.query_start_loc, db.k_pool, db.v_pool, db.block_tables,
       db.context_lens, wl.scale, maxq, workspace=ws, err=db.err)
    assert err_word(db) == 0
    return out


def _oracle(wl, causal, v_pool=None):
    fn = oracle.paged_prefill if causal else oracle.paged_cross
    return fn(wl.q, wl.query_start_loc, wl.k_pool,
              wl.v_pool if v_pool is None else v_pool, wl.block_tables,
              wl.context_lens, wl.scale)


def _slot(wl, s, j):
    ps = wl.k_pool.shape[1]
    return int(wl.block_tables[s, j // ps]), j % ps


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows", [1, 4, 8, 40, 150])
def test_two_keys_that_nearly_cancel(rows, causal):
    """Each row's weight lies on key 3 (score 0) and one more, of score -t / 64
    with t in [1/2, 3/2), whose V is the negative of key 3's; the others' scores
    are below -128, weights below e^-128, nothing in binary32.  The output
    (1 - w) / (1 + w) x has hardly a fiftieth of |x|, so a weight rounded once
    to bf16 (half a step near w is 2^-9) would show as a tenth of it.

    Bound: the output's rounding, 2^-8 of it, and for the weights 2^-15 of
    |x| = sum p |v| / sum p: 2^-16 from two bf16 terms (2^-8 x 2^-8), below
    2^-17 from the exponential (2^-18.5 by the polynomial, 2^-22 by the special
    function unit), and 2^-20 from the binary32 score, at most 8 log2 units from
    the running offset, and sums."""
    lens = [700, 2000, 600 + rows, 200 + rows]
    wl = U.cross_workload(lens, [rows] * 4, 801, num_q_heads=16,
                          num_kv_heads=4)
    rng = np.random.default_rng(rows)
    wl.scale = 0.125
    q = np.zeros(wl.q.shape, np.float32)
    q[..., 0] = rng.uniform(0.5, 1.5, q.shape[:2])
    wl.q = _bits(q)
    k = W.bf16_to_f64(wl.k_pool)
    k[..., 0] = -2048
    v = W.bf16_to_f64(wl.v_pool)
    for s, n in enumerate(lens):
        for h in range(4):
            # every place of a key in its tile comes up, first halves included
            j = (n - rows) // 2 + 13 * h + 7 * s + 16 * h * s
            a, b = _slot(wl, s, 3), _slot(wl, s, min(j, n - rows))
            k[a][h, 0] = 0
            k[b][h, 0] = -0.125
            v[b][h] = -v[a][h]
    wl.k_pool, wl.v_pool = _bits(k), _bits(v)
    ref = _oracle(wl, causal)
    size = _oracle(wl, causal, wl.v_pool & np.uint16(0x7fff))
    assert (np.abs(ref) < size / 50).all()
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * size
    for ws in (False, True):
        got = W.bf16_to_f64(bf16_bits(_run(wl, causal, ws)))
        off = np.abs(got - ref) / bound
        assert (off <= 1).all(), (ws, off.max(), (off > 1).mean())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows,lens,hidden", [
    (4, [600, 100], [200, 64]),        # 16 rows x heads: no padded row
    (8, [600, 130], [300, 90]),        # 32
    (3, [600, 100], [200, 64]),        # padded
    (70, [900, 400], [400, 130]),      # the tile kernel
    (8, [30000, 70], [14000, 20]),     # cut along the keys: parts without
    (70, [30000, 200], [14000, 64]),   # any finite score
], ids=["16", "32", "padded", "tiles", "cut", "cut tiles"])
def test_scores_of_minus_infinity_come_before_the_first_finite(rows, lens,
                                                               hidden, causal):
    """An infinity in K gives scores of minus infinity: weight zero, as long as
    some key of the row has a finite score.  What comes first in the context
    must make no difference."""
    wl = U.cross_workload(lens, [rows] * 2, 802, num_q_heads=8, num_kv_heads=2)
    q = W.bf16_to_f64(wl.q)
    q[..., 0] = np.abs(q[..., 0]) + 0.25
    wl.q = _bits(q)
    k = W.bf16_to_f64(wl.k_pool)
    for s, n in enumerate(hidden):
        for j in range(n):
            k[_slot(wl, s, j)][:, 0] = -np.inf
    wl.k_pool = _bits(k)
    ref = _oracle(wl, causal)
    for ws in (False, True):
        assert_parity(_run(wl, causal, ws), ref, f"workspace={ws}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows", [4, 8, 90])
def test_a_row_does_not_depend_on_the_rows_beside_it(rows, causal):
    """Half of the rows are made 40 times as large, so that their running
    offsets move many times and the others' warps go the longer way: the others
    keep their bits."""
    wl = U.cross_workload([1500, 300], [rows] * 2, 803, num_q_heads=8,
                          num_kv_heads=2)
    loud = np.random.default_rng(rows).random(wl.q.shape[:2]) < 0.5
    q = W.bf16_to_f64(wl.q)
    calm = [bf16_bits(_run(wl, causal, ws)) for ws in (False, True)]
    wl.q = _bits(np.where(loud[..., None], 40 * q, q))
    for ws in (False, True):
        got = bf16_bits(_run(wl, causal, ws))
        np.testing.assert_array_equal(got[~loud], calm[ws][~loud])
