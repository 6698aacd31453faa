"""One workspace of the balanced decode serves batches of any shape that it is
large enough for, in any order."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import (assert_parity, bf16_bits, err_word, gpu_append,
                      oracle_after_append, require_gpu, upload)
from paged_kv_cache_376_b200 import _lib
from paged_kv_cache_376_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _lens(n, seed, lo, hi):
    return np.random.default_rng(seed).integers(lo, hi, n).tolist()


def test_one_decode_workspace_for_every_batch():
    """Few long sequences, many, other numbers of KV heads and group sizes,
    through one buffer, each against the oracle; the counters at its front are
    zero after every call."""
    shapes = {
        "few": ([6000, 3000], 32, 8),
        "many": (_lens(64, 5, 700, 1500), 32, 8),
        "heads": (_lens(20, 6, 100, 3000), 16, 16),
        "group": (_lens(48, 7, 300, 2000), 32, 4),
        "one": ([9000], 4, 1),
    }
    cases = {}
    for i, (name, (lens, hq, hkv)) in enumerate(shapes.items()):
        wl = W.decode_workload(lens, seed=710 + i, num_q_heads=hq,
                               num_kv_heads=hkv)
        db = upload(wl)
        gpu_append(db)
        kp, vp = oracle_after_append(wl)
        cases[name] = wl, db, oracle.paged_decode(
            wl.q, kp, vp, wl.block_tables, wl.context_lens, wl.scale)
    size = max(_lib.decode_workspace(64, hq, hkv).numel()
               for _, hq, hkv in shapes.values())
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = {}
    for name in ("few", "many", "heads", "few", "group", "many", "one",
                 "heads", "group", "few", "many"):
        wl, db, ref = cases[name]
        out = torch.full_like(db.q, 7.0)
        _lib.tv_paged_decode_balanced(out, db.q, db.k_pool, db.v_pool,
                                      db.block_tables, db.context_lens,
                                      wl.scale, ws, err=db.err)
        assert err_word(db) == 0
        assert_parity(out, ref, name)
        np.testing.assert_array_equal(bf16_bits(out),
                                      first.setdefault(name, bf16_bits(out)))
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert int(ws[:4 * 16 * sms].count_nonzero()) == 0, name
