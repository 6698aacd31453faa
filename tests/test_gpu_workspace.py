"""One workspace serves calls of any shape that it is large enough for, in any
order: a server allocates it once for its largest batch, and the batch changes
from step to step.  Each call is compared with the oracle, and the counters at
the front of the buffer have to be zero after it."""
import numpy as np
import pytest
import torch

import oracle
import serving_util as U
from gpu_util import (assert_parity, bf16_bits, err_word, gpu_append,
                      oracle_after_append, require_gpu, upload)
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Case:
    """A chunk or cross-attention call and what it has to give."""

    def __init__(self, causal, lens, rows, hq, hkv, seed):
        self.causal = causal
        kw = dict(num_q_heads=hq, num_kv_heads=hkv)
        if causal:
            self.wl = W.prefill_workload([n - t for n, t in zip(lens, rows)],
                                         rows, seed=seed, **kw)
            self.db = upload(self.wl)
            gpu_append(self.db)
            kp, vp = oracle_after_append(self.wl)
            fn = oracle.paged_prefill
        else:
            self.wl = U.cross_workload(lens, rows, seed, **kw)
            self.db = upload(self.wl)
            kp, vp = self.wl.k_pool, self.wl.v_pool
            fn = oracle.paged_cross
        w = self.wl
        self.ref = fn(w.q, w.query_start_loc, kp, vp, w.block_tables,
                      w.context_lens, w.scale)
        self.maxq = max(rows)
        self.first = None

    def run(self, ws, what):
        db = self.db
        fn = (_lib.tv_paged_chunk if self.causal
              else _lib.tv_paged_cross_attention)
        out = torch.full_like(db.q, 7.0)     # rows nobody writes stand out
        fn(out, db.q, db.query_start_loc, db.k_pool, db.v_pool,
           db.block_tables, db.context_lens, self.wl.scale, self.maxq,
           workspace=ws, err=db.err)
        assert err_word(db) == 0
        assert_parity(out, self.ref, what)
        # the same call gives the same bits whatever came before it
        bits = bf16_bits(out)
        if self.first is None:
            self.first = bits
        np.testing.assert_array_equal(bits, self.first)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert int(ws[:3 * 4 * sms].count_nonzero()) == 0, what


def _lens(n, seed, lo, hi):
    return np.random.default_rng(seed).integers(lo, hi, n).tolist()


@pytest.mark.parametrize("rows", [3, 40], ids=["drafts", "prompts"])
def test_one_chunk_workspace_for_every_batch(rows):
    few = _lens(4, 1, 2000, 4000)
    many = _lens(64, 2, 700, 1500)
    mixed = [rows if s % 3 == 0 else 1 for s in range(64)]
    cases = {
        "few": Case(True, few, [rows] * 4, 32, 8, 701),
        "many": Case(True, many, mixed, 32, 8, 702),
        "cross": Case(False, _lens(40, 3, 300, 900), [1, rows] * 20, 16, 16,
                      703),
        "one head": Case(True, [9000, 50], [rows] * 2, 4, 1, 704),
    }
    ws = _lib.chunk_workspace(64, 64, 64, 16)
    for name in ("few", "many", "cross", "few", "one head", "many", "cross",
                 "one head", "many", "few"):
        cases[name].run(ws, name)


def test_a_workspace_of_the_smallest_batch_that_is_large_enough():
    """Without rows for the tile kernel the size does not depend on the number
    of sequences: a buffer made for two serves 64, and the other way round."""
    few = Case(True, [5000, 3000], [2, 4], 32, 8, 705)
    many = Case(True, _lens(64, 4, 500, 1500), [4] * 64, 32, 8, 706)
    for n in (2, 64):
        ws = _lib.chunk_workspace(n, 4, 32, 8)
        for case in (few, many, few, many):
            case.run(ws, f"sized for {n}")
