"""Inputs of the chunk, cross-attention, multi-axis rotary and pool-edit
tests (numpy; bf16 as uint16 bit patterns)."""
from __future__ import annotations

import numpy as np

from paged_kv_cache_376_b200 import workloads as W


def cross_workload(enc_lens, rows, seed, **kw):
    """Encoder states of ``enc_lens[s]`` tokens in pages (stale slots NaN) and
    ``rows[s]`` query rows per sequence."""
    wl = W.prefill_workload(enc_lens, [0] * len(enc_lens), seed=seed,
                            num_pages=max(1, sum(-(-n // kw.get("page_size", 16))
                                                 for n in enc_lens)), **kw)
    wl.q = W._normal_bf16(seed, 2, (int(sum(rows)), kw.get("num_q_heads", 32),
                                    W.HEAD_DIM))
    wl.query_start_loc = np.concatenate(
        [[0], np.cumsum(rows)]).astype(np.int32)
    return wl


def rope_table(max_position, base=500000.0):
    inv = base ** (-np.arange(32) / 32.0)
    ang = np.arange(max_position)[:, None] * inv
    return np.stack([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def multi_axis_positions(t, axes, max_position, seed):
    rng = np.random.default_rng(seed)
    return rng.integers(0, max_position, (axes, t)).astype(np.int32)


def pair_axes(axes, interleaved):
    i = np.arange(32)
    return (i % axes if interleaved else i * axes // 32).astype(np.int32)


def random_pool(seed, num_pages, batch, page_size, share=0.3, width=None):
    """Tables and lengths of a pool after a while of serving: shuffled pages,
    some sequences sharing a prefix of their left neighbour's pages."""
    rng = np.random.default_rng(seed)
    width = width or 12
    free = list(rng.permutation(num_pages))
    bt = np.full((batch, width), -1, np.int32)
    ctx = np.zeros(batch, np.int32)
    for s in range(batch):
        n = int(rng.integers(0, width + 1))
        keep = 0
        if s and rng.random() < share:
            keep = min(n, -(-int(ctx[s - 1]) // page_size))
            bt[s, :keep] = bt[s - 1, :keep]
        n = min(n, keep + len(free))
        for b in range(keep, n):
            bt[s, b] = free.pop()
        ctx[s] = max(0, n * page_size - int(rng.integers(0, page_size))) \
            if n else 0
    return bt, ctx
